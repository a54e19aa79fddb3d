"""The 8-bit pool's host side: the oracle's codes, plans for the 8-bit pool, refusals (no GPU)."""
import ctypes as C

import numpy as np
import pytest
import torch

from oracle import quantised as Q
from prefix_shared_kv_gb300 import rx, workloads as W


def test_oracle_codes_agree_with_torch():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(Q.VALUES, want)
    rng = np.random.default_rng(3)
    x = np.concatenate([rng.standard_normal(4000) * s for s in (1e-3, 0.1, 1, 30, 200)])
    grid = np.sort(Q.VALUES[np.isfinite(Q.VALUES)])
    x = np.concatenate([x, grid, (grid[1:] + grid[:-1]) / 2])  # every code and every tie
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(Q.encode(x), want)


def test_oracle_quantise_reads_back_within_half_a_step():
    rng = np.random.default_rng(4)
    bits = W.normal_bf16(rng, (50, 128))
    bits[7] = 0
    codes, scale = Q.quantise(bits)
    x = Q.A.bf16_to_f64(bits)
    err = np.abs(Q.values(codes, scale) - x)
    # half an e4m3 step: 2^-4 of the value, or half of the smallest code (2^-10) times the scale;
    # the two float32 roundings of r and x r move a value by at most 2^-23 more
    assert (err <= np.maximum(np.abs(x) * 2.0 ** -4, scale[:, None] * 2.0 ** -10) * (1 + 1e-6)).all()
    assert (np.abs(Q.VALUES[codes]).max(-1)[x.any(-1)] == 448).all()
    assert scale[7] == Q.MIN_SCALE and not codes[7].any()


def _desc(hq=8, hkv=2, pool=4096, rows=8, stride=512):
    return rx.KVDesc(hq, hkv, 128, 128 ** -0.5, pool, 0x1000, rows, stride)


def _decode_plan(kv_type, desc, seq_len, **groups):
    plan = rx.Plan()
    plan.set_kv_type(kv_type)
    rx.decode_plan(plan, desc, np.arange(len(seq_len)), seq_len, **groups)
    return plan


def test_plan_kv_type_is_checked(librx):
    plan = rx.Plan()
    for bad in (-1, 2, 77):
        with pytest.raises(rx.RxError) as e:
            plan.set_kv_type(bad)
        assert e.value.status == rx.RX_ERR_INVALID
    assert librx.rx_plan_set_kv_type(None, 0) == rx.RX_ERR_INVALID


def test_calls_of_the_other_pool_type_are_refused(librx):
    desc, kv = _desc(), rx.KVQ8(4096, 4096, 4096, 4096)
    bf, q8 = _decode_plan(rx.RX_KV_BF16, desc, [5, 9]), _decode_plan(rx.RX_KV_E4M3, desc, [5, 9])
    q8.set_kv_type(rx.RX_KV_BF16)  # for plans built from now on: the built one stays 8-bit
    with pytest.raises(rx.RxError) as e:
        rx.decode_attn_q8(bf, desc, kv, 4096, 4096, 4096, 4096, stream=0)
    assert e.value.status == rx.RX_ERR_INVALID and "bf16 pool" in str(e.value)
    with pytest.raises(rx.RxError) as e:
        rx.decode_attn(q8, desc, 4096, 4096, 4096, 4096, 4096, 4096, stream=0)
    assert e.value.status == rx.RX_ERR_INVALID and "8-bit pool" in str(e.value)
    for kv_type, call in ((rx.RX_KV_BF16, lambda p: rx.extend_attn_q8(
            p, desc, kv, 4096, 4096, 4096, 4096, stream=0)), (rx.RX_KV_E4M3, lambda p: rx.extend_attn(
            p, desc, 4096, 4096, 4096, 4096, 4096, 4096, stream=0))):
        plan = rx.Plan()
        plan.set_kv_type(kv_type)
        rx.extend_plan(plan, desc, [0, 1], [5, 9], [3, 1])
        with pytest.raises(rx.RxError) as e:
            call(plan)
        assert e.value.status == rx.RX_ERR_INVALID and "pool" in str(e.value)


def test_pair_kernel_is_refused_for_the_8_bit_pool(librx):
    plan = rx.Plan()
    plan.set_kv_type(rx.RX_KV_E4M3)
    plan.set_extend_kernel(rx.RX_EXTEND_PAIR)
    with pytest.raises(rx.RxError) as e:
        rx.extend_plan(plan, _desc(), [0], [5], [3])
    assert e.value.status == rx.RX_ERR_UNSUPPORTED
    plan.set_extend_kernel(rx.RX_EXTEND_TILES)
    rx.extend_plan(plan, _desc(), [0], [5], [3])
    assert plan.rows() == 3 and plan.launches() == 2


def test_store_and_load_refusals(librx):
    desc = _desc()
    good = rx.KVQ8(4096, 4096, 4096, 4096)

    def store(d=desc, kv=good, k=4096, v=4096, slots=4096, n=3):
        return librx.rx_store_kv_q8(C.byref(d) if d else None, C.byref(kv) if kv else None, k, v,
                                    slots, n, None)

    def load(d=desc, kv=good, k=4096, v=4096, slots=4096, n=3):
        return librx.rx_load_kv_q8(C.byref(d) if d else None, C.byref(kv) if kv else None, slots,
                                   n, k, v, None)

    bad_dim = _desc()
    bad_dim.head_dim = 64
    for call in (store, load):
        assert call(d=None) == rx.RX_ERR_INVALID
        assert call(d=bad_dim) == rx.RX_ERR_UNSUPPORTED
        assert call(kv=None) == rx.RX_ERR_INVALID
        for i in range(4):
            ptrs = [4096] * 4
            ptrs[i] = 0
            assert call(kv=rx.KVQ8(*ptrs)) == rx.RX_ERR_INVALID
            ptrs[i] = 4096 + 4
            assert call(kv=rx.KVQ8(*ptrs)) == rx.RX_ERR_INVALID
        assert call(k=0) == rx.RX_ERR_INVALID
        assert call(v=8) == rx.RX_ERR_INVALID
        assert call(slots=0) == rx.RX_ERR_INVALID
        assert call(n=-1) == rx.RX_ERR_INVALID
        assert call(n=1 << 31) == rx.RX_ERR_RANGE
        assert call(n=0) == rx.RX_OK
        assert call(n=0, kv=None, k=0, v=0, slots=0) == rx.RX_OK


def test_kv_q8_checks_its_tensors():
    code = torch.zeros(16, 2, 128, dtype=torch.uint8)
    scale = torch.zeros(16, 2)
    kv = rx.kv_q8(code, code.view(torch.float8_e4m3fn), scale, scale)
    assert kv.k_code == code.data_ptr() and kv.v_scale == scale.data_ptr()
    for bad in ((code.half(), code, scale, scale), (code, code[:8], scale, scale),
                (code, code, scale.double(), scale), (code, code, scale, scale[:, :1]),
                (code[:, :, ::2], code, scale, scale), (code[0], code[0], scale, scale),
                (code.view(torch.int8), code, scale, scale)):
        with pytest.raises(ValueError):
            rx.kv_q8(*bad)


def test_calls_check_their_tensors_against_the_pool_and_the_plan(librx):
    desc = _desc(pool=16)
    kv = rx.kv_q8(torch.zeros(16, 2, 128, dtype=torch.uint8),
                  torch.zeros(16, 2, 128, dtype=torch.uint8), torch.zeros(16, 2),
                  torch.zeros(16, 2))
    rows = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):  # host tensors are refused before anything is launched
        rx.store_kv_q8(desc, kv, rows, rows, slots, stream=0)
    with pytest.raises(ValueError):
        rx.load_kv_q8(desc, kv, slots, rows, rows, stream=0)
    with pytest.raises(ValueError):
        rx.store_kv_q8(desc, kv, rows[:2], rows, slots, stream=0)
    with pytest.raises(ValueError):
        rx.store_kv_q8(_desc(pool=17), kv, rows, rows, slots, stream=0)
    plan = _decode_plan(rx.RX_KV_E4M3, desc, [5, 9])
    o = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        rx.decode_attn_q8(plan, desc, kv, o[:1], o, torch.zeros(2, 8), 4096, stream=0)
    with pytest.raises(ValueError):
        rx.decode_attn_q8(plan, desc, kv, o, o, torch.zeros(2, 8).half(), 4096, stream=0)


@pytest.mark.parametrize("hq,hkv", [(8, 2), (32, 32), (6, 3), (8, 1), (96, 12)])
def test_decode_plan_for_the_8_bit_pool_reads_each_key_as_often_as_its_units(librx, hq, hkv):
    """A group of up to 16 stacked rows reads its prefix once; each request its own keys once."""
    gq = hq // hkv
    members = 16 // gq
    desc = _desc(hq, hkv, pool=1 << 20, rows=64, stride=4096)
    seq = [700 + 13 * b for b in range(members)] + [1, 40]
    plan = _decode_plan(rx.RX_KV_E4M3, desc, seq, group_of_req=[0] * members + [-1, -1],
                        group_prefix_len=[700])
    own = sum(13 * b for b in range(members)) + 41
    assert plan.key_reads() == (700 + own) * hkv
    assert plan.launches() == 2 and plan.rows() == members + 2


def test_decode_plan_for_very_large_groups_reads_their_prefix_once(librx):
    desc = _desc(32, 8, pool=1 << 20, rows=512, stride=4096)
    for members, reads, launches in ((16, 1, 3), (17, 2, 3), (32, 2, 3), (33, 1, 4), (300, 1, 4)):
        plan = _decode_plan(rx.RX_KV_E4M3, desc, [3000 + 10] * members,
                            group_of_req=[0] * members, group_prefix_len=[3000])
        assert plan.key_reads() == (3000 * reads + 10 * members) * 8, members
        assert plan.launches() == launches, members


def test_decode_plan_checks_are_those_of_the_bf16_pool(librx):
    desc = _desc()
    for seq in ([0], [513], [-1]):
        with pytest.raises(rx.RxError) as e:
            _decode_plan(rx.RX_KV_E4M3, desc, seq)
        assert e.value.status == rx.RX_ERR_RANGE
    empty = _decode_plan(rx.RX_KV_E4M3, desc, np.zeros(0, np.int32))
    assert empty.launches() == 0 and empty.rows() == 0


def test_extend_plan_for_the_8_bit_pool_reads_each_distinct_key_once(librx):
    """A group's prefix is expanded once for all its members and tiles, a request's own keys once;
    the workspace holds them: 64-key blocks of two 16 KiB images, two rows of scales and a word."""
    hkv, gp = 4, 300
    desc = _desc(16, hkv, pool=1 << 20, rows=64, stride=4096)
    new = [100, 1, 700, 0, 40]
    prefix = [gp, gp + 64, gp, gp, 200]
    plan = rx.Plan()
    plan.set_kv_type(rx.RX_KV_E4M3)
    rx.extend_plan(plan, desc, [0, 1, 2, 3, 4], prefix, new, [0, 0, 0, 0, -1], [gp])
    own = 100 + 65 + 700 + 240
    assert plan.key_reads() == (gp + own) * hkv
    tiles = sum(-(-n // 64) for n in (gp, 100, 65, 700, 240))
    blocks = tiles * hkv * (2 * 64 * 256 + 2 * 64 * 4 + 128)
    # (and, the batch being small, at most one partial pair of tiles of 128 rows per SM)
    assert blocks <= plan.workspace_size() <= blocks + 160 * 256 * 516 + 65536
    bf = rx.Plan()
    rx.extend_plan(bf, desc, [0, 1, 2, 3, 4], prefix, new, [0, 0, 0, 0, -1], [gp])
    assert bf.workspace_size() < 65536 and bf.launches() == 1


def test_extend_plan_of_few_new_tokens_needs_no_expansion(librx):
    """One or two new tokens a request on long prefixes: planned as a decode of them, whose workspace
    holds partial rows only.  The row count is the new tokens' all the same, and the plan serves
    extend calls only."""
    plan = rx.Plan()
    plan.set_kv_type(rx.RX_KV_E4M3)
    desc = _desc(32, 8, pool=1 << 20, rows=64, stride=8192)
    new = [1, 2, 0, 1]
    rx.extend_plan(plan, desc, [0, 1, 2, 3], [5000] * 4, new, [0, 0, 0, -1], [4000])
    assert plan.rows() == 4 and plan.launches() == 2
    # the group's prefix; the first's and the last's keys past it; the second's cached keys, and its
    # new tokens' own
    assert plan.key_reads() == (4000 + 1001 + 5001 + 1000 + 1 + 2) * 8
    assert plan.workspace_size() < 1 << 23
    with pytest.raises(rx.RxError) as e:
        rx.decode_attn_q8(plan, desc, rx.KVQ8(4096, 4096, 4096, 4096), 4096, 4096, 4096, 4096,
                          stream=0)
    assert e.value.status == rx.RX_ERR_INVALID and "built for extend" in str(e.value)
    rx.extend_plan(plan, desc, [0, 1, 2, 3], [5000] * 4, [200] * 4, [0, 0, 0, -1], [4000])
    assert plan.workspace_size() > (4000 + 3 * 1000 + 5000) * 8 * 512


def test_extend_plan_splits_the_keys_of_a_batch_too_small_for_the_gpu(librx):
    """Four requests of 40 new tokens on 1,000 cached ones: five tiles a head would leave most SMs
    idle, so the tiles' keys are split and a merge is launched; a batch that fills the GPU is not."""
    plan = rx.Plan()
    plan.set_kv_type(rx.RX_KV_E4M3)
    desc = _desc(8, 2, pool=1 << 20, rows=64, stride=4096)
    rx.extend_plan(plan, desc, [0, 1, 2, 3], [1000] * 4, [40] * 4, [0] * 4, [1000])
    assert plan.launches() == 3 and plan.rows() == 160
    assert plan.key_reads() == (1000 + 160) * 2
    desc = _desc(32, 32, pool=1 << 20, rows=64, stride=4096)
    rx.extend_plan(plan, desc, np.arange(32), [1000] * 32, [200] * 32)
    assert plan.launches() == 2


@pytest.mark.parametrize("new", [[], [0], [0, 0]])
def test_calls_without_rows_take_no_tensors(librx, new):
    """A plan without work enqueues nothing: its call may be given NULL tensors and pools, and still
    needs the right plan, descriptor and workspace."""
    desc = _desc()
    null, part = rx.KVQ8(0, 0, 0, 0), rx.KVQ8(4096, 0, 4096, 8)
    for kv_type in (rx.RX_KV_BF16, rx.RX_KV_E4M3):
        plan = rx.Plan()
        plan.set_kv_type(kv_type)
        if new:
            rx.extend_plan(plan, desc, np.arange(len(new)), [5] * len(new), new)
            bf16, q8 = librx.rx_extend_attn, librx.rx_extend_attn_q8
        else:
            rx.decode_plan(plan, desc, np.zeros(0, np.int32), np.zeros(0, np.int32))
            bf16, q8 = librx.rx_decode_attn, librx.rx_decode_attn_q8
        for ws, size, status in ((0x1000, 1 << 20, rx.RX_OK), (0x1000, 8, rx.RX_ERR_WORKSPACE),
                                 (None, 1 << 20, rx.RX_ERR_WORKSPACE),
                                 (0x1010, 1 << 20, rx.RX_ERR_INVALID)):
            if kv_type == rx.RX_KV_BF16:
                # (RX_ERR_CUDA: past the checks, the kernels' attributes need a GPU)
                got = bf16(plan.handle, C.byref(desc), None, None, None, None, None, ws, size, None)
                assert got == status or (status == rx.RX_OK and got == rx.RX_ERR_CUDA)
                assert q8(plan.handle, C.byref(desc), None, None, None, None, ws, size,
                          None) == rx.RX_ERR_INVALID
            else:
                for kv in (None, C.byref(null), C.byref(part)):
                    assert q8(plan.handle, C.byref(desc), kv, None, None, None, ws, size,
                              None) == status
    plan = _decode_plan(rx.RX_KV_E4M3, desc, [5])  # with rows every pointer is looked at
    for kv in (None, C.byref(null), C.byref(part)):
        assert librx.rx_decode_attn_q8(plan.handle, C.byref(desc), kv, 4096, 4096, 4096, 0x1000,
                                       1 << 30, None) == rx.RX_ERR_INVALID


def test_the_current_stream_is_found_without_torchs_private_call(monkeypatch):
    class Stream:
        cuda_stream = 77

    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(rx, "_torch_calls", None, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream)
    assert rx._stream(None) == 77 and rx._stream(5) == 5 and rx._stream(Stream) == 77
