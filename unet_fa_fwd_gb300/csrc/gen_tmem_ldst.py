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
out = []
for n in (8, 16, 32, 64, 128):
    out.append(ld(n))
for n in (8, 16, 32):
    out.append(st(n))
open(os.path.join(os.path.dirname(os.path.abspath(__file__)), "tmem_ldst.inc"), "w").write(
"// Long-hand tcgen05.ld / tcgen05.st wrappers (32x32b shape: thread t of warp w\n"
"// addresses TMEM lane 32*(w%4)+t).  Each load waits (tcgen05.wait::ld) inside the\n"
"// same asm statement, so no use of the outputs can be scheduled before the wait.\n"
"// The instructions are .sync.aligned: every lane of the warp must execute them\n"
"// together, so each wrapper first reconverges the warp (__syncwarp) -- after a\n"
"// branch the compiler cannot prove uniform, the warp may otherwise still be split.\n"
"// Generated by gen_tmem_ldst.py; included by sm100_ptx.cuh only.\n\n" + "\n".join(out))
