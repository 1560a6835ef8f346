"""Writes tmem_ldst.inc: the long-hand tcgen05.ld / tcgen05.st wrappers.

Run ``python gen_tmem_ldst.py`` in this directory after editing; the
generated file is part of the sources.
"""
import os

def ld(n):
    regs = ",".join(f"%{i}" for i in range(n))
    outs = ", ".join(f'"=r"(r[{i}])' for i in range(n))
    return f'''// {n} consecutive 32-bit TMEM columns of this thread's lane, waited for.
__device__ __forceinline__ void tmem_ld32x32b_x{n}(uint32_t taddr, uint32_t (&r)[{n}]) {{
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x{n}.b32 {{{regs}}}, [%{n}];\\n"
      "tcgen05.wait::ld.sync.aligned;\\n"
      : {outs}
      : "r"(taddr)
      : "memory");
}}
'''
def st(n):
    regs = ",".join(f"%{i+1}" for i in range(n))
    ins = ", ".join(f'"r"(r[{i}])' for i in range(n))
    return f'''// Store {n} consecutive 32-bit TMEM columns of this thread's lane (not waited for).
__device__ __forceinline__ void tmem_st32x32b_x{n}(uint32_t taddr, const uint32_t (&r)[{n}]) {{
  __syncwarp();
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x{n}.b32 [%0], {{{regs}}};\\n"
      :
      : "r"(taddr), {ins}
      : "memory");
}}
'''
SHAPES = {
    # 16 columns of the warp's 32 lanes: (name, what, [(shape, lane offset, elements' places)])
    "row": ("r[c] is this thread's lane, column c", [("32x32b.x16", 0, list(range(16)))]),
    "quad": ("r[8 i + 2 j + c] is lane t / 4 + 8 j, column 8 i + 2 (t % 4) + c",
             [("16x256b.x2", 16 * h, [8 * (k // 4) + 4 * h + k % 4 for k in range(8)]) for h in (0, 1)]),
}
STORES = {
    "quad": ("r[4 i + j] is lane t / 4 + 8 j, column 4 i + t % 4",
             [("16x128b.x2", 16 * h, [4 * (k // 2) + 2 * h + k % 2 for k in range(4)]) for h in (0, 1)]),
}
def ld16(name, arrays):
    """16 consecutive columns at each of `arrays` addresses, waited for once."""
    what, parts = SHAPES[name]
    outs, ins, lines = [], [], []
    n = 16 * arrays
    for a in range(arrays):
        outs += [f'"=r"({"rs"[a]}[{i}])' for i in range(16)]
        for shape, lane, at in parts:
            regs = ",".join(f"%{16 * a + i}" for i in at)
            lines.append(f'"tcgen05.ld.sync.aligned.{shape}.b32 {{{regs}}}, [%{n + len(ins)}];\\n"')
            t = "taddr" if a == 0 else "saddr"
            ins.append(f'"r"({t} + ({lane}u << 16))' if lane else f'"r"({t})')
    body = "\n      ".join(lines)
    two = arrays == 2
    return f'''// 16 consecutive 32-bit TMEM columns of the warp's 32 lanes{" at each address" if two else ""}, waited for:
// {what}.
__device__ __forceinline__ void tmem_ld_{name}16{"_two" if two else ""}(uint32_t taddr, uint32_t (&r)[16]{", uint32_t saddr, uint32_t (&s)[16]" if two else ""}) {{
  __syncwarp();
  asm volatile(
      {body}
      "tcgen05.wait::ld.sync.aligned;\\n"
      : {", ".join(outs)}
      : {", ".join(ins)}
      : "memory");
}}
'''
def st8(name):
    what, parts = STORES[name]
    lines, addr = [], []
    for i, (shape, lane, at) in enumerate(parts):
        regs = ",".join(f"%{len(parts) + k}" for k in at)
        lines.append(f'"tcgen05.st.sync.aligned.{shape}.b32 [%{i}], {{{regs}}};\\n"')
        addr.append(f'"r"(taddr + ({lane}u << 16))' if lane else '"r"(taddr)')
    body = "\n      ".join(lines)
    ins = ", ".join(f'"r"(r[{i}])' for i in range(8))
    return f'''// Store 8 consecutive 32-bit TMEM columns of the warp's 32 lanes (not waited for):
// {what}.
__device__ __forceinline__ void tmem_st_{name}8(uint32_t taddr, const uint32_t (&r)[8]) {{
  __syncwarp();
  asm volatile(
      {body}
      :
      : {", ".join(addr)}, {ins}
      : "memory");
}}
'''
out = []
for n in (8, 16, 32, 64, 128):
    out.append(ld(n))
for n in (8, 16, 32):
    out.append(st(n))
out += [ld16("row", 2), ld16("quad", 1), ld16("quad", 2), st8("quad")]
open(os.path.join(os.path.dirname(os.path.abspath(__file__)), "tmem_ldst.inc"), "w").write(
"// Long-hand tcgen05.ld / tcgen05.st wrappers (32x32b shape: thread t of warp w\n"
"// addresses TMEM lane 32*(w%4)+t).  Each load waits (tcgen05.wait::ld) inside the\n"
"// same asm statement, so no use of the outputs can be scheduled before the wait.\n"
"// The instructions are .sync.aligned: every lane of the warp must execute them\n"
"// together, so each wrapper first reconverges the warp (__syncwarp) -- after a\n"
"// branch the compiler cannot prove uniform, the warp may otherwise still be split.\n"
"// Generated by gen_tmem_ldst.py; included by sm100_ptx.cuh only.\n\n" + "\n".join(out))
