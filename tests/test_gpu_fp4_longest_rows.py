"""4-bit casts of the longest rows that an int32 counts: K padded to a multiple of 256 is 2^31 there."""
import numpy as np
import pytest
import torch

from tests import _block_quant as bq
from tests._gpu import bf16_bits, u8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [bq.MXFP4, bq.NVFP4])
def test_cast_of_a_row_just_below_2_31(cuda_lib, kind):
    """Codes and scales of the row's end, zero bytes where K is padded and in the rows that fill up the atoms."""
    cols = (1 << 31) - 96
    part = torch.randn(1 << 20, generator=torch.Generator().manual_seed(kind)).to(torch.bfloat16).cuda()
    x = part.repeat(2048)[:cols].view(1, cols)
    q = torch.empty(1, cols // 2, dtype=torch.uint8, device="cuda")
    sf = torch.full((cuda_lib.fp4_scale_bytes(1, cols, kind),), 0xFF, dtype=torch.uint8, device="cuda")
    scale = dict(scale=torch.full((1,), 100.0, device="cuda")) if kind == bq.NVFP4 else {}
    cuda_lib.fp4_cast_multi([dict(x=x, quant=kind, q_row=q, sf_row=sf, **scale)])
    torch.cuda.synchronize()
    cuda_lib.fp8t_check_device_error()
    n, tail = {bq.MXFP4: 32, bq.NVFP4: 16}[kind], 4096 - 96
    codes, s = bq.quantise(bf16_bits(x[:, -tail:].contiguous()), kind, 100.0)
    assert np.array_equal(bq.unpack(u8(q[:, -tail // 2:])), codes)
    atoms = sf.view(-1, 512)                             # row 0's four scales of an atom are its first word
    last = u8(atoms[-(4096 // n // 4):, :4].contiguous()).reshape(-1)
    assert np.array_equal(last[:tail // n], s[0]) and not last[tail // n:].any()
    assert all(int(a[:, 4:].max()) == 0 for a in atoms.split(1 << 20))
