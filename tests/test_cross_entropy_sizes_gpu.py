"""linear_cross_entropy and its gradient at the largest vocabulary that a call takes,
where the end of the last piece is past 2**31, and of most tokens (needs a GB300 and about 40 GB of free
device memory).

One input of one token makes the logits the weights themselves, w of 33 values: the sum
of exponentials is that of how often each occurs.  Bounds as in test_cross_entropy_gpu:
2**-21 of each exponential; the additions' roundings, 16 in a thread and those of up to 2**25
parts by 1024 at a time, 2**15 in order, each part joined by a product and a sum (2**16 counted);
of a bf16 gradient its own rounding and that of dz, 2**-8 each, and of its exponent, at most 34
in powers of two, two roundings."""
import pytest

torch = pytest.importorskip("torch")

import dense_fp32_tiled_gb300 as sg

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def test_the_last_piece_of_the_largest_vocabulary():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_fp32_tiled_gb300 import build
    build.build()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB free on the device")
    N = 2147480000  # 64 pieces of 2**25 columns end at 2**31
    w = torch.empty((1, N), dtype=torch.bfloat16, device="cuda")
    values = (torch.arange(33, device="cuda") / 8 - 2).to(torch.bfloat16)
    count = torch.zeros(33, dtype=torch.float64, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for a in range(0, N, 1 << 28):
        at = torch.randint(0, 33, (min(1 << 28, N - a),), generator=g, device="cuda", dtype=torch.uint8)
        for k in range(33):
            count[k] += (at == k).sum()
        for b in range(0, len(at), 1 << 26):
            w[0, a + b:a + b + (1 << 26)] = values[at[b:b + (1 << 26)].long()]
    target = N - 3
    x, targets = torch.ones((1, 1), dtype=torch.bfloat16, device="cuda"), torch.tensor([target], device="cuda")
    loss, lse = sg.linear_cross_entropy(x, w, targets)
    e = torch.exp(values.double())
    want = torch.log((count * e).sum())
    assert abs(float(lse) - float(want)) <= 2.0 ** -21 + 2 ** 16 * U + 4 * U * float(want)
    assert abs(float(loss) - float(want) + float(w[0, target])) <= 2.0 ** -21 + 2 ** 16 * U + 8 * U * float(want)
    dx, dw = sg.linear_cross_entropy_backward(torch.ones(1, device="cuda"), x, w, targets, lse)
    p = torch.exp(values.double() - lse.double())
    goal = (count * p * values.double()).sum() - w[0, target].double()
    # each product's dz rounded by 2**-9, and the sum of 2**25 columns in pieces and shares by the tensor
    # cores, which cut: all of one kind cancel against nothing, so the magnitudes' sum bounds it
    size = (count * p * values.double().abs()).sum() + w[0, target].double().abs()
    assert abs(float(dx) - float(goal)) <= float((2.0 ** -8 + 2.0 ** -6) * size)
    for a in list(range(0, N, 1 << 25)) + [N - 4096]:  # where pieces begin, and the end
        for lo in (max(0, a - 600), a):
            r = slice(lo, min(N, lo + 600 if lo == a else a))
            z = w[0, r].double()
            ref = torch.exp(z - lse.double())
            bound = ref * (2.0 ** -7 + 2.0 ** -17)
            if r.start <= target < r.stop:
                ref[target - r.start] -= 1
                bound[target - r.start] += 2.0 ** -8
            assert ((dw[0, r].double() - ref).abs() <= bound).all(), (r.start, r.stop)
    assert float(dw[0, target]) < -0.9
    assert sg.linear_timeouts() == 0


def test_the_last_of_the_most_tokens():
    # (about 110 GB of device memory)  One column and a gradient of the log sum alone: dz is 1, dx the weight.
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_fp32_tiled_gb300 import build
    build.build()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 140 << 30:
        pytest.skip("needs 140 GiB free on the device")
    M = 2147480000  # a step of the blocks that look after the tokens is 152 * 1024
    x = torch.ones((M, 1), dtype=torch.bfloat16, device="cuda")
    w = torch.full((1, 1), 1.5, dtype=torch.bfloat16, device="cuda")
    targets = torch.zeros(M, dtype=torch.int32, device="cuda")
    lse, dlse = torch.full((M,), 1.5, device="cuda"), torch.ones(M, device="cuda")
    dlse[-1] = 0.5
    dx, dw = sg.linear_cross_entropy_backward(None, x, w, targets, lse, dlse=dlse, need_dw=False)
    assert dw is None and dx.shape == (M, 1)
    for a in range(0, M, 1 << 28):
        part = dx[a:a + (1 << 28), 0]
        if a + (1 << 28) >= M:
            assert float(part[-1]) == 0.75
            part = part[:-1]
        assert (part == 1.5).all()
    assert sg.linear_timeouts() == 0
    del x, targets, lse, dlse, dx, part
    torch.cuda.empty_cache()
