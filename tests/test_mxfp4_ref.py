"""Pins of the plain MXFP4 forms (tests/mxfp4_ref.py): worked cases of the OCP
rule, a brute-force nearest value, and the block and packing layouts."""
import torch

import mxfp4_ref as ref


def row(*values):
    v = torch.zeros(32, dtype=torch.float64)
    v[:len(values)] = torch.tensor(values, dtype=torch.float64)
    return v


def test_worked_blocks():
    # amax 6: scale 1, every value of the format is itself
    v = row(*ref.GRID.tolist(), *(-ref.GRID).tolist())
    codes, scales = ref.quantize(v)
    assert scales.tolist() == [127]
    assert (codes & 15)[:8].tolist() == [0, 2, 4, 6, 8, 10, 12, 14] and (codes >> 4)[:8].tolist() == [1, 3, 5, 7, 9, 11, 13, 15]
    assert torch.equal(ref.dequantize(codes, scales), v)
    # ties go to the even code: 1/4 -> 0, 3/4 -> 1, 5/4 -> 1, 7/4 -> 2, 5/2 -> 2, 7/2 -> 4, 5 -> 4; 7 saturates
    v = row(6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 7)
    assert ref.dequantize(*ref.quantize(v))[1:9].tolist() == [0, 1, 1, 2, 2, 4, 4, 6]
    # amax 1: scale 2^-2
    codes, scales = ref.quantize(row(1.0, 0.3))
    assert scales.tolist() == [125] and ref.dequantize(codes, scales)[:2].tolist() == [1.0, 0.25]
    # a zero block, and one below the smallest scale
    assert ref.quantize(row())[1].tolist() == [0]
    codes, scales = ref.quantize(row(2.0 ** -130))
    assert scales.tolist() == [0] and ref.dequantize(codes, scales)[0] == 0
    # Inf and NaN make the whole block NaN
    for bad in (float("inf"), float("nan")):
        codes, scales = ref.quantize(row(1.0, bad))
        assert scales.tolist() == [255] and not codes.any() and ref.dequantize(codes, scales).isnan().all()


def test_rounding_is_nearest():
    g = torch.Generator().manual_seed(3)
    a = torch.rand(4096, generator=g, dtype=torch.float64) * 6
    d = (a.unsqueeze(1) - ref.GRID).abs()
    assert torch.equal((ref.GRID[ref.round_codes(a)] - a).abs(), d.min(1).values)


def test_blocks_and_packing_round_trip():
    g = torch.Generator().manual_seed(4)
    for E, rows, K in ((2, 64, 512), (1, 32, 256), (3, 32, 640)):
        codes = torch.randint(0, 256, (E, rows, K // 2), generator=g, dtype=torch.uint8)
        scales = torch.randint(0, 256, (E, rows, K // 32), generator=g, dtype=torch.uint8)
        G, units = ref.group_of(K), K // 128
        packed = torch.zeros(E * rows // 16, units * 1088, dtype=torch.uint8)
        for e in range(E):           # the layout, byte by byte
            for r in range(rows):
                blk = (e * rows + r) // 32 * 2 + (r % 8) // 4
                m = 4 * (r % 32 // 8) + r % 4
                for u in range(units):
                    base = u // G * G * 1088
                    for kb in range(4):
                        at = base + u % G * 1024 + 16 * (16 * kb + m)
                        packed[blk, at:at + 16] = codes[e, r, u * 64 + kb * 16:u * 64 + kb * 16 + 16]
                        packed[blk, base + G * 1024 + G * (16 * kb + m) + u % G] = scales[e, r, u * 4 + kb]
        c, s = ref.unpack_weights(packed, E, rows, K)
        assert torch.equal(c, codes) and torch.equal(s, scales)
