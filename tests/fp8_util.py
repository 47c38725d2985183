"""Inputs and comparisons shared by the GPU tests of the 8-bit operators."""
import numpy as np
import torch

from software_pipelined_tiled_02_amd import binding
from tests import fp8_ref as R

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
NAN_BYTE = 0x7F            # a NaN in both 8-bit types


def f8_of(raw, fp8):
    return torch.from_numpy(np.ascontiguousarray(raw)).cuda().view(F8[fp8])


def raw_of(t):
    return t.view(torch.uint8).cpu().numpy()


def values(rng, m, k, spread=0.5):
    return (rng.standard_normal((m, k)) * np.exp(spread * rng.standard_normal((1, k)))).astype(np.float32)


def operand(rng, rows, k, fp8, scale_rows):
    """A quantised matrix of normal values: (bit patterns, fp32 scales)."""
    return R.quantize_fp32(values(rng, rows, k) * np.float32(0.1 + rng.random()), fp8, scale_rows)


def place_bytes(raw, ld, offset):
    """Bytes on the GPU with rows `ld` apart from byte `offset` of a buffer of
    NaNs that ends with the last row's last byte; returns the matrix."""
    rows, k = raw.shape
    flat = np.full(max(1, offset + (rows - 1) * ld + k), NAN_BYTE, dtype=np.uint8)
    for r in range(rows):
        flat[offset + r * ld:offset + r * ld + k] = raw[r]
    return torch.from_numpy(flat).cuda()[offset:].as_strided((rows, k), (ld, 1))


def check_product(c, a, sa, b, sb, at, bt, rows, out, what, base=None):
    """C (a tensor) against the definition; base: what an accumulating call started from."""
    ref, path, instr = R.product(R.decode(a, at), sa.astype(np.float64), R.decode(b, bt), sb.astype(np.float64), rows)
    off = path if out == "f32" else path + instr
    if base is not None:
        ref = ref + base
        off = off + np.abs(ref) * R.U
    R.assert_within(c.double().cpu().numpy(), ref, off + R.half_step(np.abs(ref) + off, out), what)


def run_product(a, sa, b, sb, at, bt, **kw):
    """binding.run_fp8 on operands whose rows start on 16 bytes, NaNs between them."""
    k = a.shape[1]
    ld = -(-max(k, 1) // 16) * 16
    return binding.run_fp8(place_bytes(a, ld, 0).view(F8[at]), torch.from_numpy(sa).cuda(),
                           place_bytes(b, ld, 0).view(F8[bt]), torch.from_numpy(sb).cuda(), **kw)
