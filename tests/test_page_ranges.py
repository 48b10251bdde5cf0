"""kv_attend_pages on the tensor cores where magnitudes lie apart or end: keys far above the
others under values of any size, tokens behind a row's position, values at both ends of the
range that the header states, infinities in pages and windows. Against 64-bit attention over
the dequantized values; TOL_TENSOR as derived in test_pages.py (six roundings of 2^-11), which
holds wherever probabilities and scales keep their 11 bits.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import kvq_oracle as O  # noqa: E402
from test_pages import TOL_F32, TOL_TENSOR, attention64, kvq  # noqa: E402,F401
from test_pages_edges import check_rows, one_request  # noqa: E402


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("each_warp", [False, True])
@pytest.mark.parametrize("size", [0.05, 1.0, 30.0, 500.0, 3000.0, 1e5])
def test_keys_far_above_the_others(kvq, d, each_warp, size):  # noqa: F811
    # Sink keys 11.5 nats above the rest, with zero values, one or one in each of the groups of
    # an item: the output is the others', which keep 11 bits down to 11.8 nats below. Channel 0
    # alone makes the sinks' scores, so that the others differ by a tenth of a nat at most.
    # A sink's score is one product of three factors rounded to 11 bits (q times the scale, the K
    # scale, their product; 2^-11 each, relative): 11.5 * 3 * 2^-11 = 0.017 nats. It scales the
    # sum of the probabilities, and with it all of the output alike, by no more than 1.7 %; what
    # is left of the difference without that common factor is the others' own, TOL_TENSOR.
    gen = torch.Generator(device="cuda").manual_seed(d + int(size))
    n = 512
    sinks = [5, 41, 77, 124] if each_warp else [77]
    q = torch.randn((2, 8, d), generator=gen, device="cuda") * 0.02
    q[:, :, 0] = 4.0
    k = torch.randn((n, 1, d), generator=gen, device="cuda")
    k[:, :, 0] = 0.0
    k[sinks, 0, 0] = 11.5 * d ** 0.5 / 4.0
    v = torch.randn((n, 1, d), generator=gen, device="cuda") * size
    v[sinks] = 0.0
    q, k, v = q.bfloat16(), k.bfloat16(), v.bfloat16()
    cache, values = one_request(kvq, n, k, v, 0, 1, d)
    a = np.einsum("td,rhd->rht", values[0][0], q.double().cpu().numpy()) / np.sqrt(d)
    rest = np.delete(a, sinks, axis=2)
    gap = a[:, :, sinks].max(2) - rest.min(2), a[:, :, sinks].min(2) - rest.max(2)
    assert gap[0].max() < 11.8 and gap[1].min() > 11.0
    call = kvq.AttendPages(cache, q, torch.zeros(2, dtype=torch.int32, device="cuda"),
                           out_dtype="f32")
    got = call.run().double().cpu().numpy()
    assert kvq.read_status(call.status) == 0 and call.path == "pages_tensor"
    for i in range(2):
        want = attention64(q[i].double().cpu().numpy(), *values)
        for h in range(8):
            common = (got[i, h] @ want[h]) / (want[h] @ want[h])
            assert abs(common - 1.0) <= 0.017 + TOL_TENSOR, (i, h)
            assert O.rel_l2(got[i, h], common * want[h]) <= TOL_TENSOR, (i, h)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1e3, 1e7, 1e9, 1e15, float("inf"), float("-inf"), float("nan")])
def test_tokens_behind_the_position_have_no_part(kvq, d, size):  # noqa: F811
    # rows that end inside an int4 group and inside a window tile, whose later tokens have
    # values of another size: what they see is as if the request ended there
    gen = torch.Generator(device="cuda").manual_seed(d)
    n, window = 640, 96
    for last in (489, 481, 510, 575, 600):
        k = torch.randn((n, 1, d), generator=gen, device="cuda")
        v = torch.randn((n, 1, d), generator=gen, device="cuda")
        v[last + 1:] = size
        k, v = k.bfloat16(), v.bfloat16()
        q = torch.randn((1, 8, d), generator=gen, device="cuda").bfloat16()
        with np.errstate(all="ignore"):
            cache, (kk, vv) = one_request(kvq, n, k, v, window, 1, d)
        call = kvq.AttendPages(cache, q, torch.zeros(1, dtype=torch.int32, device="cuda"),
                               torch.full((1,), last, dtype=torch.int32, device="cuda"),
                               out_dtype="f32")
        got = call.run().double().cpu().numpy()
        assert kvq.read_status(call.status) == 0 and call.path == "pages_tensor"
        want = attention64(q[0].double().cpu().numpy(), kk[:, :last + 1], vv[:, :last + 1])
        assert O.rel_l2(got[0], want) <= TOL_TENSOR, last


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1e-16, 1e-12, 1e-9, 1e10, 1e13, 1e16, 1e17])
@pytest.mark.parametrize("window", [0, 64])
def test_values_at_the_ends_of_the_range(kvq, d, size, window):  # noqa: F811
    gen = torch.Generator(device="cuda").manual_seed(d)
    n = 640
    k = torch.randn((n, 1, d), generator=gen, device="cuda").bfloat16()
    v = (torch.randn((n, 1, d), generator=gen, device="cuda") * size).bfloat16()
    # (every group's largest value is within the header's 2.4e-17 and 5e17)
    most = v.abs().view(n, d // 32, 32).amax(-1)
    assert 2.4e-17 < float(most.min()) and float(most.max()) < 5e17
    cache, values = one_request(kvq, n, k, v, window, 1, d)
    q = torch.randn((3, 8, d), generator=gen, device="cuda").bfloat16()
    check_rows(kvq, cache, values, q, TOL_TENSOR)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_both_ends_in_one_request(kvq, d):  # noqa: F811
    # the sum of the probabilities keeps the weight of groups whose values do not show
    gen = torch.Generator(device="cuda").manual_seed(d)
    n = 1024
    size = torch.ones(n, device="cuda")
    size[:300], size[300:332], size[400:500], size[700:710] = 1e-16, 0.0, 1e-8, 1e17
    k = torch.randn((n, 1, d), generator=gen, device="cuda").bfloat16()
    v = (torch.randn((n, 1, d), generator=gen, device="cuda") * size[:, None, None]).bfloat16()
    for order in (slice(None), torch.arange(n - 1, -1, -1, device="cuda")):
        cache, values = one_request(kvq, n, k[order], v[order], 64, 1, d)
        q = torch.randn((2, 8, d), generator=gen, device="cuda").bfloat16()
        check_rows(kvq, cache, values, q, TOL_TENSOR)


@pytest.mark.gpu
@pytest.mark.parametrize("d,wdt", [(64, "bf16"), (128, "bf16"), (96, "f32")])
@pytest.mark.parametrize("size", [float("inf"), float("-inf"), 1e30])
def test_infinite_values_in_the_pages_stay_in_their_features(kvq, d, wdt, size):  # noqa: F811
    # an infinite value's group has an infinite scale and code 0: NaN for its 32 features, and
    # nothing else. (On the tensor cores a scale of 2^56 and more counts as one.)
    gen = torch.Generator(device="cuda").manual_seed(d)
    n = 320
    k = torch.randn((n, 2, d), generator=gen, device="cuda").bfloat16()
    v = torch.randn((n, 2, d), generator=gen, device="cuda").bfloat16()
    v[77, 1, 40] = size
    v[200, 1, 33] = -size
    q = torch.randn((3, 8, d), generator=gen, device="cuda").bfloat16()
    with np.errstate(all="ignore"):
        cache, (kk, vv) = one_request(kvq, n, k, v, 0, 2, d, wdt)
    vv[:, :, 32:64] = 0.0
    call = kvq.AttendPages(cache, q, torch.zeros(3, dtype=torch.int32, device="cuda"),
                           torch.tensor([n - 1, 76, 150], dtype=torch.int32, device="cuda"),
                           out_dtype="f32")
    got = call.run().double().cpu().numpy()
    assert kvq.read_status(call.status) == 0
    for i, m in enumerate((n, 77, 151)):
        want = attention64(q[i].double().cpu().numpy(), kk[:, :m], vv[:, :m])
        bad = np.zeros((8, d), bool)
        if m > 77 and (wdt == "bf16" or np.isinf(size)):
            bad[4:, 32:64] = True
        assert (np.isnan(got[i])[:, 32:64] == bad[:, 32:64]).all(), i
        got[i][:, 32:64] = 0.0
        assert O.rel_l2(got[i], want) <= (TOL_TENSOR if wdt == "bf16" else TOL_F32), i


def with_infinities(d, wdt, gen):
    """Window keys and values with infinities under queries of known signs; what the 64-bit
    definition makes of them."""
    n, window = 200, 100
    k = torch.randn((n, 1, d), generator=gen, device="cuda").bfloat16()
    v = torch.randn((n, 1, d), generator=gen, device="cuda").bfloat16()
    q = torch.randn((1, 4, d), generator=gen, device="cuda").bfloat16()
    return n, window, k, v, q


@pytest.mark.gpu
@pytest.mark.parametrize("d,wdt", [(64, "bf16"), (128, "bf16"), (96, "f32"), (96, "bf16")])
@pytest.mark.parametrize("at", [100, 130, 199])
def test_infinite_values_in_the_window(kvq, d, wdt, at):  # noqa: F811
    gen = torch.Generator(device="cuda").manual_seed(d + at)
    n, window, k, v, q = with_infinities(d, wdt, gen)
    v[at, 0, 3], v[at, 0, 9] = float("inf"), float("-inf")
    v[at, 0, 20], v[at - 3 if at > 100 else at + 3, 0, 20] = float("inf"), float("-inf")
    cache, (kk, vv) = one_request(kvq, n, k, v, window, 1, d, wdt)
    out, status = kvq.attend_pages(cache, q, torch.zeros(1, dtype=torch.int32, device="cuda"),
                                   out_dtype="f32")
    assert kvq.read_status(status) == 0
    got = out[0].double().cpu().numpy()
    assert (got[:, 3] == np.inf).all() and (got[:, 9] == -np.inf).all()
    assert np.isnan(got[:, 20]).all()
    keep = [i for i in range(d) if i not in (3, 9, 20)]
    want = attention64(q[0].double().cpu().numpy(), kk, np.where(np.isfinite(vv), vv, 0.0))
    assert O.rel_l2(got[:, keep], want[:, keep]) <= (TOL_TENSOR if wdt == "bf16" else TOL_F32)


@pytest.mark.gpu
@pytest.mark.parametrize("d,wdt", [(64, "bf16"), (128, "bf16"), (96, "f32"), (96, "bf16")])
@pytest.mark.parametrize("at", [100, 130, 199])
@pytest.mark.parametrize("same", [False, True])
def test_infinite_keys_in_the_window(kvq, d, wdt, at, same):  # noqa: F811
    # a score of -inf leaves the token out, one of +inf or of both infinities has no softmax
    gen = torch.Generator(device="cuda").manual_seed(d + at)
    n, window, k, v, q = with_infinities(d, wdt, gen)
    q[0, :, 5] = torch.tensor([1.0, -1.0, 0.37, -1e-3], device="cuda").bfloat16()
    q[0, :, 17] = q[0, :, 5] if same else -q[0, :, 5]
    k[at, 0, 5], k[at, 0, 17] = float("-inf"), float("-inf")
    cache, (kk, vv) = one_request(kvq, n, k, v, window, 1, d, wdt)
    out, status = kvq.attend_pages(cache, q, torch.zeros(1, dtype=torch.int32, device="cuda"),
                                   out_dtype="f32")
    assert kvq.read_status(status) == 0
    got = out[0].double().cpu().numpy()
    rest = np.delete(np.arange(n), at)
    want = attention64(q[0].double().cpu().numpy(), kk[:, rest], vv[:, rest])
    for h in range(4):
        if same and h in (0, 2):
            assert O.rel_l2(got[h], want[h]) <= (TOL_TENSOR if wdt == "bf16" else TOL_F32), h
        else:
            assert np.isnan(got[h]).all(), h


@pytest.mark.gpu
@pytest.mark.parametrize("d,wdt", [(64, "bf16"), (128, "bf16"), (96, "f32"), (96, "bf16")])
def test_a_row_whose_scores_are_all_minus_infinity_is_zero(kvq, d, wdt):  # noqa: F811
    gen = torch.Generator(device="cuda").manual_seed(d)
    n = 45
    k = torch.randn((n, 1, d), generator=gen, device="cuda").bfloat16()
    v = torch.randn((n, 1, d), generator=gen, device="cuda").bfloat16()
    q = torch.randn((2, 2, d), generator=gen, device="cuda").bfloat16()
    q[:, 0, 7], q[:, 1, 7] = 0.5, -0.5
    k[:, 0, 7] = float("-inf")
    cache, _ = one_request(kvq, n, k, v, 100, 1, d, wdt)
    out, status = kvq.attend_pages(cache, q, torch.zeros(2, dtype=torch.int32, device="cuda"),
                                   torch.tensor([n - 1, 3], dtype=torch.int32, device="cuda"),
                                   out_dtype="f32")
    assert kvq.read_status(status) == 0
    assert bool((out[:, 0] == 0).all()) and bool(out[:, 1].isnan().all())


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [100, 3900])
@pytest.mark.parametrize("size", [1e-25, 1e25, 1e36])
def test_values_of_any_magnitude_in_the_window(kvq, d, n, size):  # noqa: F811
    # (one CTA's unit, and one whose partials are joined)
    gen = torch.Generator(device="cuda").manual_seed(d + n)
    k = torch.randn((n, 1, d), generator=gen, device="cuda").bfloat16()
    v = (torch.randn((n, 1, d), generator=gen, device="cuda") * size).bfloat16()
    cache, values = one_request(kvq, n, k, v, 4000, 1, d)
    q = torch.randn((2, 8, d), generator=gen, device="cuda").bfloat16()
    check_rows(kvq, cache, values, q, TOL_TENSOR)
