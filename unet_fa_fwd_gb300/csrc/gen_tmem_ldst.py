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
def ld2(n):
    """Two loads of 16 lanes by 256 bits: an element's place is 8 * (8-column block) + 2 * (row / 8) + its column."""
    at = [[8 * (k // 4) + 4 * h + k % 4 for k in range(4 * n)] for h in (0, 1)]
    # (early-clobber: the first load's results must not take the register of the second one's address)
    outs = ", ".join(f'"=&r"(r[{i}])' for i in range(8 * n))
    lines = "\n      ".join(f'"tcgen05.ld.sync.aligned.16x256b.x{n}.b32 {{{{{",".join(f"%{i}" for i in at[h])}}}}}, [%{8 * n + h}];\\n"'
                             for h in (0, 1)).replace("{{", "{").replace("}}", "}")
    return f'''// {8 * n} consecutive 32-bit TMEM columns of the warp's 32 lanes, waited for: r[8 i + 2 j + c]
// is lane t / 4 + 8 j, column 8 i + 2 (t % 4) + c.
__device__ __forceinline__ void tmem_ld2x16x256b_x{n}(uint32_t taddr, uint32_t (&r)[{8 * n}]) {{
  __syncwarp();
  asm volatile(
      {lines}
      "tcgen05.wait::ld.sync.aligned;\\n"
      : {outs}
      : "r"(taddr), "r"(taddr + (16u << 16))
      : "memory");
}}
'''
def st2(n):
    """The same pairs of columns, packed in one: two stores of 16 lanes by 128 bits."""
    at = [[4 * (k // 2) + 2 * h + k % 2 + 2 for k in range(2 * n)] for h in (0, 1)]
    ins = ", ".join(f'"r"(r[{i}])' for i in range(4 * n))
    lines = "\n      ".join(f'"tcgen05.st.sync.aligned.16x128b.x{n}.b32 [%{h}], {{{{{",".join(f"%{i}" for i in at[h])}}}}};\\n"'
                             for h in (0, 1)).replace("{{", "{").replace("}}", "}")
    return f'''// Store {4 * n} consecutive 32-bit TMEM columns of the warp's 32 lanes (not waited for): r[4 i + j]
// is lane t / 4 + 8 j, column 4 i + t % 4.
__device__ __forceinline__ void tmem_st2x16x128b_x{n}(uint32_t taddr, const uint32_t (&r)[{4 * n}]) {{
  __syncwarp();
  asm volatile(
      {lines}
      :
      : "r"(taddr), "r"(taddr + (16u << 16)), {ins}
      : "memory");
}}
'''
out = []
for n in (8, 16, 32, 64, 128):
    out.append(ld(n))
for n in (8, 16, 32):
    out.append(st(n))
out.append(ld2(1))
out.append(ld2(4))
out.append(st2(4))
open(os.path.join(os.path.dirname(os.path.abspath(__file__)), "tmem_ldst.inc"), "w").write(
"// Long-hand tcgen05.ld / tcgen05.st wrappers (32x32b shape: thread t of warp w\n"
"// addresses TMEM lane 32*(w%4)+t).  Each load waits (tcgen05.wait::ld) inside the\n"
"// same asm statement, so no use of the outputs can be scheduled before the wait.\n"
"// The instructions are .sync.aligned: every lane of the warp must execute them\n"
"// together, so each wrapper first reconverges the warp (__syncwarp) -- after a\n"
"// branch the compiler cannot prove uniform, the warp may otherwise still be split.\n"
"// Generated by gen_tmem_ldst.py; included by sm100_ptx.cuh only.\n\n" + "\n".join(out))
