"""CPU tests of norm_quantize, the block product and sampling: what they
refuse, and empty calls, which return before any HIP call.  Device addresses are
plain integers."""

import pytest

import gemm_rwkv_amd.rq as rq

BASE = 0x7f0000000000
STEP = 0x10000000        # room between two fake buffers
A = [BASE + i * STEP for i in range(16)]
B128 = rq.RQ_FP8_E4M3_B128

# dtype, norm, x, delta, alpha, rows, width, ld, gamma, beta, eps, fmt, x_out, codes, scales
NORM = [rq.RQ_F16, rq.RQ_NORM_LAYER, A[0], A[1], 1.0, 10, 256, 264, A[2], A[3], 1e-5, B128, A[4], A[5], A[6]]
# xq, sx, m, w, dtype, y, ldy
GEMM = [A[0], A[1], 10, (B128, 0, 200, 256, A[2], A[3]), rq.RQ_F16, A[4], 200]
# dtype, logits, rows, vocab, ld, temperature, top_k, top_p, min_p, u, token, logprob
SAMPLE = [rq.RQ_F32, A[0], 10, 100, 104, A[1], A[2], A[3], A[4], A[5], A[6], A[7]]


def _call(fn, args, changed=(), **kw):
    a = list(args)
    for i, v in dict(changed).items():
        a[i] = v
    if fn is rq.rq_gemm_fp8_block:
        a[3] = rq.QWeight(*a[3])
    return fn(*a, **kw)


def _status(fn, args, changed, **kw):
    with pytest.raises(rq.RqError) as e:
        _call(fn, args, changed, **kw)
    return e.value.status


CALLS = [(rq.rq_norm_quantize, NORM, [2, 13, 14], [2, 3, 8, 9, 12, 13, 14]), (rq.rq_gemm_fp8_block, GEMM, [0, 1, 5], [0, 1, 5]),
         (rq.rq_sample, SAMPLE, [1, 9, 10], [1])]
IDS = [c[0].__name__ for c in CALLS]


@pytest.mark.parametrize("fn,args,needed,aligned", CALLS, ids=IDS)
def test_pointers(fn, args, needed, aligned):
    for at in needed:
        assert _status(fn, args, {at: None}) == rq.RQ_ERR_NULL, at
    for at in aligned:
        assert _status(fn, args, {at: args[at] + 8}) == rq.RQ_ERR_ALIGN, at


def test_sample_rows_are_of_four_bytes():
    for at in (5, 6, 7, 8, 9, 10, 11):
        assert _status(rq.rq_sample, SAMPLE, {at: SAMPLE[at] + 2}) == rq.RQ_ERR_ALIGN
    # a slice of a longer array is fine, which the next check shows
    assert _status(rq.rq_sample, SAMPLE, {5: SAMPLE[5] + 4, 2: -1}) == rq.RQ_ERR_SHAPE


def test_weight_format():
    assert rq.rq_qweight_bytes(B128, 0, 200, 256) == (200 * 256, 2 * 4, 0, 0)
    assert rq.rq_qweight_bytes(B128, 7, 128, 640) == (128 * 640, 8, 0, 0)
    assert rq.block_scale_row(512) == 4 and rq.block_scale_row(640) == 8
    with pytest.raises(rq.RqError) as e:
        rq.rq_qweight_bytes(B128, 0, 4, 192)
    assert e.value.status == rq.RQ_ERR_SHAPE
    with pytest.raises(rq.RqError) as e:
        rq.rq_qweight_bytes(rq.RQ_F32, 0, 4, 128)
    assert e.value.status == rq.RQ_ERR_FORMAT
    w = (B128, 0, 200, 256, None, A[3])
    assert _status(rq.rq_gemm_fp8_block, GEMM, {3: w}) == rq.RQ_ERR_NULL
    assert _status(rq.rq_gemm_fp8_block, GEMM, {3: (B128, 0, 200, 256, A[2], None)}) == rq.RQ_ERR_NULL
    assert _status(rq.rq_gemm_fp8_block, GEMM, {3: (B128, 0, 200, 256, A[2], A[3] + 8)}) == rq.RQ_ERR_ALIGN
    # its codes are of one product only
    other = rq.QWeight(B128, 0, 200, 256, A[2], A[3])
    for call in (lambda: rq.rq_gemm_small_m(A[0], 4, 256, other, A[4], 200, ws=False),
                 lambda: rq.rq_gemm_fp8(A[0], A[1], 4, other, A[4], 200, ws=False),
                 lambda: rq.rq_quantize_act(A[0], 4, 256, 256, B128, A[1], A[2])):
        with pytest.raises(rq.RqError) as e:
            call()
        assert e.value.status == rq.RQ_ERR_FORMAT
    assert _status(rq.rq_gemm_fp8_block, GEMM, {3: (rq.RQ_FP8_E4M3_CH, 0, 200, 256, A[2], A[3])}) == rq.RQ_ERR_FORMAT


@pytest.mark.parametrize("changed,status", [
    ({0: rq.RQ_F32}, rq.RQ_ERR_FORMAT), ({0: 0}, rq.RQ_ERR_FORMAT), ({11: rq.RQ_F16}, rq.RQ_ERR_FORMAT), ({1: 3}, rq.RQ_ERR_VALUE),
    ({1: -1}, rq.RQ_ERR_VALUE), ({10: -1e-9}, rq.RQ_ERR_VALUE), ({10: float("nan")}, rq.RQ_ERR_VALUE),
    ({10: float("inf")}, rq.RQ_ERR_VALUE), ({5: -1}, rq.RQ_ERR_SHAPE), ({6: 192, 7: 192}, rq.RQ_ERR_SHAPE),
    ({6: 0}, rq.RQ_ERR_SHAPE), ({7: 248}, rq.RQ_ERR_SHAPE), ({7: 260}, rq.RQ_ERR_ALIGN), ({6: 16512, 7: 16512}, rq.RQ_ERR_SHAPE),
    ({11: rq.RQ_I8_CH, 6: 24}, rq.RQ_ERR_SHAPE), ({11: rq.RQ_FP8_E4M3_CH, 6: 8}, rq.RQ_ERR_SHAPE),
    ({5: 2 ** 31}, rq.RQ_ERR_SHAPE), ({5: 2 ** 30, 7: 2 ** 12}, rq.RQ_ERR_SHAPE)])
def test_norm_refusals(changed, status):
    assert _status(rq.rq_norm_quantize, NORM, changed) == status


@pytest.mark.parametrize("changed,status", [
    ({4: rq.RQ_I8_CH}, rq.RQ_ERR_FORMAT), ({2: -1}, rq.RQ_ERR_SHAPE), ({2: 2 ** 21}, rq.RQ_ERR_SHAPE), ({6: 199}, rq.RQ_ERR_SHAPE),
    ({6: 2 ** 31}, rq.RQ_ERR_SHAPE), ({3: (B128, 0, 2 ** 27 + 1, 256, A[2], A[3]), 6: 2 ** 27 + 1}, rq.RQ_ERR_SHAPE),
    ({3: (B128, 0, 200, 200, A[2], A[3])}, rq.RQ_ERR_SHAPE)])
def test_gemm_refusals(changed, status):
    assert _status(rq.rq_gemm_fp8_block, GEMM, changed) == status


@pytest.mark.parametrize("changed,status", [
    ({0: B128}, rq.RQ_ERR_FORMAT), ({2: -1}, rq.RQ_ERR_SHAPE), ({2: 2 ** 21}, rq.RQ_ERR_SHAPE), ({3: 0}, rq.RQ_ERR_SHAPE),
    ({3: 2 ** 20 + 1, 4: 2 ** 20 + 8}, rq.RQ_ERR_SHAPE), ({4: 96}, rq.RQ_ERR_SHAPE), ({4: 100}, rq.RQ_ERR_ALIGN)])
def test_sample_refusals(changed, status):
    assert _status(rq.rq_sample, SAMPLE, changed) == status


@pytest.mark.parametrize("fn,args,outs,ins", [(rq.rq_norm_quantize, NORM, [12, 13, 14], [2, 3, 8, 9]),
                                              (rq.rq_gemm_fp8_block, GEMM, [5], [0, 1]),
                                              (rq.rq_sample, SAMPLE, [10, 11], [1, 5, 6, 7, 8, 9])], ids=IDS)
def test_outputs_overlap_nothing(fn, args, outs, ins):
    for o in outs:
        for i in ins + [z for z in outs if z != o]:
            if fn is rq.rq_norm_quantize and (o, i) == (12, 2):
                continue       # x_out may be x
            assert _status(fn, args, {o: args[i]}) == rq.RQ_ERR_ALIAS, (o, i)
    if fn is rq.rq_norm_quantize:
        assert _status(fn, args, {12: args[2] + 16}) == rq.RQ_ERR_ALIAS
    if fn is rq.rq_gemm_fp8_block:
        assert _status(fn, args, {5: A[2]}) == rq.RQ_ERR_ALIAS
        assert _status(fn, args, {5: A[3]}) == rq.RQ_ERR_ALIAS


def test_empty_calls():
    _call(rq.rq_norm_quantize, NORM, {5: 0})
    _call(rq.rq_norm_quantize, NORM, {5: 0, 2: None, 13: None, 14: None})
    _call(rq.rq_gemm_fp8_block, GEMM, {2: 0})
    _call(rq.rq_gemm_fp8_block, GEMM, {2: 0, 0: None, 1: None, 5: None})
    _call(rq.rq_gemm_fp8_block, GEMM, {3: (B128, 0, 0, 256, A[2], A[3]), 6: 1})
    _call(rq.rq_sample, SAMPLE, {2: 0})
    _call(rq.rq_sample, SAMPLE, {2: 0, 1: None, 9: None, 10: None})
