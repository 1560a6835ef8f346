"""Writes mma_batch.inc: the batched tcgen05.mma issue wrappers.

Each wrapper issues n MMAs of one tile from a single inline-asm block with the
operand-address offsets as immediates.  Run ``python gen_mma_batch.py`` in this
directory after editing; the generated file is part of the sources.
"""
import os
def ss(n, kind, elect=False):
    tparams = ", ".join(f"int O{i}" for i in range(1, n))
    g = "@e " if elect else ""
    lines = ['"{\\n"', '".reg .pred p, q;\\n"', '".reg .b32 al, bl;\\n"', '".reg .b64 da, db;\\n"']
    if elect:
        lines += ['".reg .pred e;\\n"', '".reg .b32 el;\\n"', '"elect.sync el|e, 0xffffffff;\\n"']
    lines += ['"setp.ne.b32 p, %6, 0;\\n"', '"setp.eq.u32 q, 0, 0;\\n"',
              '"mov.b64 da, {%1, %2};\\n"', '"mov.b64 db, {%3, %4};\\n"',
              f'"{g}tcgen05.mma.cta_group::1.kind::{kind} [%0], da, db, %5, p;\\n"']
    for i in range(1, n):
        op = 6 + i
        lines += [f'"add.u32 al, %1, %{op};\\n"', f'"add.u32 bl, %3, %{op};\\n"',
                  '"mov.b64 da, {al, %2};\\n"', '"mov.b64 db, {bl, %4};\\n"',
                  f'"{g}tcgen05.mma.cta_group::1.kind::{kind} [%0], da, db, %5, q;\\n"']
    lines.append('"}\\n"')
    imm = "".join(f', "n"(O{i})' for i in range(1, n))
    name = f"mma_ss{'_f8' if kind != 'f16' else ''}_x{n}{'_el' if elect else ''}"
    tmpl = f"template <{tparams}>\n" if n > 1 else ""
    body = "\n      ".join(lines)
    return f'''{tmpl}__device__ __forceinline__ void {name}(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                          uint32_t b_hi, uint32_t idesc, uint32_t acc_first) {{
  asm volatile(
      {body}
      ::"r"(d), "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc_first){imm}
      : "memory");
}}
'''
def ts(n, elect=False):
    g = "@e " if elect else ""
    lines = ['"{\\n"', '".reg .pred p, q;\\n"', '".reg .b32 ta, bl;\\n"', '".reg .b64 db;\\n"']
    if elect:
        lines += ['".reg .pred e;\\n"', '".reg .b32 el;\\n"', '"elect.sync el|e, 0xffffffff;\\n"']
    lines += ['"setp.ne.b32 p, %5, 0;\\n"', '"setp.eq.u32 q, 0, 0;\\n"',
              '"mov.b64 db, {%2, %3};\\n"',
              f'"{g}tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\\n"']
    for i in range(1, n):
        lines += [f'"add.u32 ta, %1, {8 * i};\\n"', f'"add.u32 bl, %2, %{5 + i};\\n"',
                  '"mov.b64 db, {bl, %3};\\n"',
                  f'"{g}tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], db, %4, q;\\n"']
    lines.append('"}\\n"')
    body = "\n      ".join(lines)
    imm = "".join(f', "n"(BSTEP * {i})' for i in range(1, n))
    return f'''template <int BSTEP>
__device__ __forceinline__ void mma_ts_x{n}{'_el' if elect else ''}(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi,
                                          uint32_t idesc, uint32_t acc_first) {{
  asm volatile(
      {body}
      ::"r"(d), "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc_first){imm}
      : "memory");
}}
'''
out = ["// Batched tcgen05.mma issue: n MMAs of one tile in a single asm block, so the\n"
       "// issuer spends two 32-bit adds per MMA on operand addresses (the offsets\n"
       "// are immediates) and sets its predicates once.  The first MMA accumulates\n"
       "// iff acc_first != 0, the others always accumulate.  Descriptors are given\n"
       "// as 32-bit halves; the start address is in the low half.  Called by a\n"
       "// converged warp with warp-uniform operands: elect.sync picks one lane,\n"
       "// which issues the MMAs (the *_el suffix).\n"
       "// Generated by gen_mma_batch.py; included by sm100_ptx.cuh only.\n"]
for n in (1, 2, 4, 8):
    out.append(ss(n, "f16", True))
for n in (1, 2, 4):
    out.append(ss(n, "f8f6f4", True))
out.append(ts(4, True))
out.append(ts(8, True))
open(os.path.join(os.path.dirname(os.path.abspath(__file__)), "mma_batch.inc"), "w").write("\n".join(out))
