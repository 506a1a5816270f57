"""CPU tests of the time-mix entry points: what they refuse, and empty calls,
which return before any HIP call.  Device addresses are plain integers."""

import pytest

import gemm_rwkv_amd.rq as rq

BASE = 0x7f0000000000
STEP = 0x10000000        # room between two fake buffers
A = [BASE + i * STEP for i in range(40)]
WS = (BASE + 0x100 * STEP, 1 << 20)
F16, BF16 = rq.RQ_F16, rq.RQ_BF16


def _status(fn, args, changed, **kw):
    a = list(args)
    for i, v in changed.items():
        a[i] = v
    with pytest.raises(rq.RqError) as e:
        fn(*a, **kw)
    return e.value.status


# dtype, r, w, k, v, a, b, tokens, heads, ld, cu, nseq, state_in, state_out, slots, nslots, y, ldy
MIX = [F16, *A[0:6], 10, 2, 128, A[6], 3, A[7], A[8], A[9], 4, A[10], 128]
# dtype, r..b, tokens, heads, ld, cu, nseq, state_in, dy, dstate_out, dr..db, dstate_in
BACK = [F16, *A[0:6], 10, 2, 128, A[6], 3, A[7], A[8], A[9], *A[10:16], A[16]]
# dtype, x, delta, alpha, tokens, width, ld, cu, nseq, gamma, beta, eps, mu, nmix, shift_in, shift_out, slots, nslots, x_out, out, ldo
NORM = [F16, A[0], A[1], 1.0, 10, 64, 64, A[2], 3, A[3], A[4], 1e-5, A[5], 6, A[6], A[7], A[8], 4, A[9], A[10], 64]
# dtype, x, alpha, tokens, width, ld, cu, nseq, gamma, beta, eps, mu, nmix, shift_in, dout, ldo, dx_out, dshift_out, dx, ddelta, dshift_in, dgamma, dbeta, dmu
NORM_BACK = [F16, A[0], 1.0, 10, 64, 64, A[1], 3, A[2], A[3], 1e-5, A[4], 6, A[5], A[6], 64, A[7], A[8], A[9], A[10], A[11],
             A[12], A[13], A[14]]
# dtype, y, r, k, v, g, tokens, heads, ld, gamma, beta, eps, u, out, ldo
GATE = [F16, *A[0:5], 10, 2, 128, A[5], A[6], 1e-5, A[7], A[8], 128]
# ..., u, dout, dy, dr, dk, dv, dg, dgamma, dbeta, du
GATE_BACK = [F16, *A[0:5], 10, 2, 128, A[5], A[6], 1e-5, A[7], A[8], *A[9:14], A[14], A[15], A[16]]

# every pointer that may not be NULL
NEEDED = [(rq.rq_time_mix, MIX, [1, 2, 3, 4, 5, 6, 16]), (rq.rq_time_mix_backward, BACK, [1, 2, 3, 4, 5, 6, 13, 15, 16, 17, 18, 19, 20]),
          (rq.rq_shift_norm, NORM, [1, 9, 10, 12, 19]), (rq.rq_shift_norm_backward, NORM_BACK, [1, 8, 9, 11, 14, 18, 21, 22, 23]),
          (rq.rq_head_gate, GATE, [1, 2, 3, 4, 5, 9, 10, 12, 13]),
          (rq.rq_head_gate_backward, GATE_BACK, [1, 2, 3, 4, 5, 9, 10, 12, 13, 14, 15, 16, 17, 18, 19, 20, 21])]
# those and the optional ones, all 16-byte aligned
ALIGNED = [NEEDED[0][2] + [12, 13], NEEDED[1][2] + [12, 14, 21], NEEDED[2][2] + [2, 14, 15, 18],
           NEEDED[3][2] + [13, 16, 17, 19, 20], NEEDED[4][2], NEEDED[5][2]]
IDS = [fn.__name__ for fn, _, _ in NEEDED]


@pytest.mark.parametrize("i", range(6), ids=IDS)
def test_pointers(i):
    fn, args, needed = NEEDED[i]
    for at in needed:
        assert _status(fn, args, {at: 0}) == rq.RQ_ERR_NULL, at
        assert _status(fn, args, {at: None}) == rq.RQ_ERR_NULL, at
    for at in ALIGNED[i]:
        assert _status(fn, args, {at: args[at] + 8}) == rq.RQ_ERR_ALIGN, at


@pytest.mark.parametrize("i", range(6), ids=IDS)
def test_outputs_overlap_nothing(i):
    fn, args, needed = NEEDED[i]
    outs = {0: [13, 16], 1: [15, 16, 17, 18, 19, 20, 21], 2: [15, 18, 19], 3: [18, 19, 20, 21, 22, 23], 4: [13],
            5: [14, 15, 16, 17, 18, 19, 20, 21]}[i]
    for at in outs:
        assert _status(fn, args, {at: args[1] + 16}) == rq.RQ_ERR_ALIAS, at      # inside the first input
        for other in outs:
            if other != at:
                assert _status(fn, args, {at: args[other]}) == rq.RQ_ERR_ALIAS, (at, other)
    if fn in (rq.rq_time_mix, rq.rq_time_mix_backward, rq.rq_shift_norm_backward, rq.rq_head_gate_backward):
        assert _status(fn, args, {}, ws=(args[1], 1 << 17)) == rq.RQ_ERR_ALIAS
        assert _status(fn, args, {}, ws=(WS[0] + 4, 1 << 17)) == rq.RQ_ERR_ALIGN
    # in place is allowed for the carried state only, and only as a whole
    if fn is rq.rq_time_mix:
        assert _status(fn, args, {13: args[12] + 16}) == rq.RQ_ERR_ALIAS
    if fn is rq.rq_shift_norm:
        assert _status(fn, args, {15: args[14] + 16}) == rq.RQ_ERR_ALIAS


@pytest.mark.parametrize("i", range(6), ids=IDS)
def test_types_and_shapes(i):
    fn, args, _ = NEEDED[i]
    tokens, width, ld = {0: (7, 8, 9), 1: (7, 8, 9), 2: (4, 5, 6), 3: (3, 4, 5), 4: (6, 7, 8), 5: (6, 7, 8)}[i]
    for bad in (0, rq.RQ_W4_SYM, rq.RQ_FP8_E4M3_CH, 99):
        assert _status(fn, args, {0: bad}) == rq.RQ_ERR_FORMAT
    assert _status(fn, args, {tokens: -1}) == rq.RQ_ERR_SHAPE
    assert _status(fn, args, {tokens: 1 << 31}) == rq.RQ_ERR_SHAPE
    assert _status(fn, args, {width: 0}) == rq.RQ_ERR_SHAPE
    assert _status(fn, args, {ld: args[ld] - 8}) == rq.RQ_ERR_SHAPE
    assert _status(fn, args, {ld: args[ld] + 4}) == rq.RQ_ERR_ALIGN
    assert _status(fn, args, {ld: 1 << 31}) == rq.RQ_ERR_SHAPE


def test_sequences_and_slots():
    for fn, args, cu, nseq in ((rq.rq_time_mix, MIX, 10, 11), (rq.rq_time_mix_backward, BACK, 10, 11),
                               (rq.rq_shift_norm, NORM, 7, 8), (rq.rq_shift_norm_backward, NORM_BACK, 6, 7)):
        assert _status(fn, args, {cu: None}) == rq.RQ_ERR_SHAPE                # 10 tokens in 3 equal sequences
        assert _status(fn, args, {nseq: 0}) == rq.RQ_ERR_SHAPE                 # tokens in no sequence
        assert _status(fn, args, {nseq: -1}) == rq.RQ_ERR_SHAPE
        assert _status(fn, args, {nseq: 1 << 23}) == rq.RQ_ERR_SHAPE
        assert _status(fn, args, {cu: args[cu] + 2}) == rq.RQ_ERR_ALIGN
    for fn, args, slots in ((rq.rq_time_mix, MIX, 14), (rq.rq_shift_norm, NORM, 16)):
        assert _status(fn, args, {slots: args[slots] + 2}) == rq.RQ_ERR_ALIGN
        assert _status(fn, args, {slots: None, slots + 1: 2}) == rq.RQ_ERR_SHAPE   # three sequences, two entries
        assert _status(fn, args, {slots + 1: -1}) == rq.RQ_ERR_SHAPE
    assert _status(rq.rq_time_mix, MIX, {17: 120}) == rq.RQ_ERR_SHAPE
    assert _status(rq.rq_time_mix, MIX, {17: 132}) == rq.RQ_ERR_ALIGN
    assert _status(rq.rq_time_mix, MIX, {8: 1 << 20, 9: 1 << 26}) == rq.RQ_ERR_SHAPE    # 2^22 heads' workgroups and rows
    assert _status(rq.rq_head_gate, GATE, {14: 120}) == rq.RQ_ERR_SHAPE


def test_norm_arguments():
    for fn, args, width, eps, nmix, ldo in ((rq.rq_shift_norm, NORM, 5, 11, 13, 20), (rq.rq_shift_norm_backward, NORM_BACK, 4, 10, 12, 15)):
        assert _status(fn, args, {nmix: 0}) == rq.RQ_ERR_SHAPE
        assert _status(fn, args, {nmix: 9}) == rq.RQ_ERR_SHAPE
        assert _status(fn, args, {width: 60}) == rq.RQ_ERR_ALIGN
        assert _status(fn, args, {width: 8200, width + 1: 8200, ldo: 8200}) == rq.RQ_ERR_SHAPE
        assert _status(fn, args, {ldo: 56}) == rq.RQ_ERR_SHAPE
        assert _status(fn, args, {ldo: 68}) == rq.RQ_ERR_ALIGN
        for bad in (-1e-5, float("nan"), float("inf")):
            assert _status(fn, args, {eps: bad}) == rq.RQ_ERR_VALUE
    for fn, args in ((rq.rq_head_gate, GATE), (rq.rq_head_gate_backward, GATE_BACK)):
        assert _status(fn, args, {11: float("nan")}) == rq.RQ_ERR_VALUE


def test_workspace_sizes():
    need = rq.rq_time_mix_backward_bytes(10, 2, 3)
    assert need > 64 << 10
    assert rq.rq_time_mix_backward_bytes(1000, 2, 3) > need
    for bad in ((-1, 2, 3), (10, 0, 3), (10, 2, -1), (1 << 31, 2, 3), (10, 2, 1 << 23)):
        assert rq.rq_time_mix_backward_bytes(*bad) == 0
    assert _status(rq.rq_time_mix_backward, BACK, {}, ws=(WS[0], need - 16)) == rq.RQ_ERR_WORKSPACE
    assert _status(rq.rq_time_mix_backward, BACK, {}, ws=False) == rq.RQ_ERR_WORKSPACE


def test_empty_calls():
    none = dict.fromkeys((12, 13, 14))
    rq.rq_time_mix(*[none.get(i, v) if i in none else (0 if i == 7 else v) for i, v in enumerate(MIX)])     # no tokens, no state
    rq.rq_time_mix(*[{7: 0, 10: None, 11: 0}.get(i, v) for i, v in enumerate(MIX)])                         # no sequences
    rq.rq_time_mix_backward(*[{7: 0, 10: None, 11: 0}.get(i, v) for i, v in enumerate(BACK)])
    rq.rq_shift_norm(*[{4: 0, 7: None, 8: 0}.get(i, v) for i, v in enumerate(NORM)])
    rq.rq_head_gate(*[0 if i == 6 else v for i, v in enumerate(GATE)])


def test_status_texts():
    for st in (rq.RQ_ERR_WORKSPACE, rq.RQ_ERR_VALUE):
        assert rq.status_str(st) != "unknown status"
