"""GPU parity of gdn_beam_select and gdn_beam_reorder against their plain references: tokens and parents equal,
scores within the derived bound, states bit-equal; and what masks, ties, ended beams, odd sizes and strides do."""
import numpy as np
import pytest
import torch

import beam_reference as ref
import ssm_recurrent_decode_gb300 as gdn

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _run(logits, scores, K, *, rows=None, finished=None, eos=-1, err=None, out_finished=None):
    batch, beams = scores.shape
    out = (torch.full((batch, K), float("nan"), device="cuda"), torch.full((batch, K), -7, dtype=torch.int32, device="cuda"),
           torch.full((batch, K), -7, dtype=torch.int32, device="cuda"))
    ws = gdn.beam_select_workspace(batch, beams, logits.shape[1], K)
    ws.fill_(0xFF)
    put = lambda a, t: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(t).cuda()
    gdn.gdn_beam_select(logits, put(scores, torch.float32), *out, rows=put(rows, torch.int32), finished=put(finished, torch.uint8),
                        eos_token=eos, workspace=ws, err_flags=err, out_finished=out_finished)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in out]


def _check(logits, scores, K, premise=True, **kw):
    got = _run(logits, scores, K, **kw)
    x = logits.float().cpu().numpy().astype(np.float64)
    s, p, t, margins = ref.select(x, scores.astype(np.float32).astype(np.float64), K,
                                  **{k: v for k, v in kw.items() if k in ("rows", "finished", "eos")})
    if premise:
        assert ref.clear(margins), "the inputs leave a choice to rounding"
    np.testing.assert_array_equal(got[1], p)
    np.testing.assert_array_equal(got[2], t)
    fin = np.isfinite(s)
    np.testing.assert_array_equal(np.isfinite(got[0]), fin)
    assert np.all(np.abs(got[0][fin] - s[fin]) <= ref.LSE_BOUND + 2.0 ** -24 * np.abs(s[fin]))
    return got


def _logits(R, V, dtype, seed, scale=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(R, V, generator=g, device="cuda")).to(TYPES[dtype])


def _scores(batch, beams, seed):
    return -np.sort(np.random.default_rng(seed).uniform(0, 20, size=(batch, beams)), axis=1).astype(np.float32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 1000, 4095, 4096, 4097, 8193, 32000, 50021])
def test_vocabulary_sizes(V, dtype):
    _check(_logits(12, V, dtype, V), _scores(3, 4, V), 8)


@pytest.mark.parametrize("batch,beams,K", [(1, 1, 1), (1, 32, 64), (5, 3, 1), (2, 16, 32), (3, 5, 64), (40, 2, 4)])
def test_beam_counts(batch, beams, K):
    _check(_logits(batch * beams, 9001, "bf16", K), _scores(batch, beams, K), K)


def test_many_segments_and_chunks():
    """One row over 32 segments of several chunks each, and many rows of one segment."""
    _check(_logits(1, 1_200_000, "bf16", 1), _scores(1, 1, 1), 16)
    _check(_logits(1, 1_200_001, "f32", 2), _scores(1, 1, 2), 16)
    _check(_logits(1300, 20000, "bf16", 3), _scores(325, 4, 3), 8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_by_index_and_strides(dtype):
    wide = _logits(20, 5003, dtype, 4)
    rows = np.random.default_rng(4).permutation(20)[:12].reshape(3, 4)
    _check(wide[:, 1:4800], _scores(3, 4, 4), 6, rows=rows)


@pytest.mark.parametrize("share", [0.5, 0.9, 0.999, 1.0])
def test_forbidden_tokens(share):
    x = _logits(8, 6000, "f32", 5)
    x[torch.rand(8, 6000, generator=torch.Generator().manual_seed(5)).cuda() < share] = -float("inf")
    x[3] = -float("inf")                       # a row without any token
    x[5, ::2] = float("nan")
    got = _check(x, _scores(2, 4, 5), 12)
    if share == 1.0:
        assert np.all(got[1] == -1) and np.all(got[2] == -1) and np.all(got[0] == -np.inf)


def test_infinite_logits_share_the_row():
    x = _logits(2, 3000, "f32", 6)
    x[0, 100] = x[0, 2000] = float("inf")
    got = _check(x, np.array([[0.0, -1.0]], dtype=np.float32), 4)
    assert got[2][0, 0] == 100 and got[2][0, 1] == 2000 and abs(got[0][0, 0] + np.log(2.0)) < 1e-6


def test_dead_and_ended_beams():
    x = _logits(12, 3000, "bf16", 7)
    s = _scores(3, 4, 7)
    s[0, 1:] = -np.inf                         # a search's first step: one beam
    s[1] = -np.inf                             # nothing at all
    s[2, 2] = np.nan
    x[4:8] = float("nan")
    _check(x, s, 6)
    fin = np.zeros((3, 4), dtype=np.uint8)
    fin[0, 0] = fin[2, 0] = fin[2, 1] = 1
    flags = torch.full((3, 6), 9, dtype=torch.uint8, device="cuda")
    got = _check(x, s, 6, finished=fin, eos=2, out_finished=flags)
    np.testing.assert_array_equal(flags.cpu().numpy(), (got[2] == 2).astype(np.uint8))
    assert list(got[1][0]) == [0, -1, -1, -1, -1, -1]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [300, 20000, 20003])
def test_equal_logits_go_by_index(V, dtype):
    """Rows of one value, the order reversed or rising, and equal beams: ties to the lower beam, then token."""
    x = torch.zeros(4, V, dtype=TYPES[dtype], device="cuda")
    got = _check(x, np.zeros((1, 4), dtype=np.float32), 10)
    assert list(got[1][0]) == [0] * 10 and list(got[2][0]) == list(range(10))
    x = torch.zeros(4, V, dtype=TYPES[dtype], device="cuda")
    x[:, 0], x[:, -1] = -0.0, 0.0
    assert list(_run(x, np.zeros((1, 4), dtype=np.float32), 3)[2][0]) == [0, 1, 2]
    ramp = (torch.arange(V, device="cuda") * (20.0 / V)).to(TYPES[dtype]).repeat(4, 1)
    _check(ramp, np.zeros((1, 4), dtype=np.float32), 9)
    _check(ramp.flip(1).contiguous(), np.zeros((1, 4), dtype=np.float32), 9)
    same = _logits(1, V, dtype, V).repeat(4, 1)
    got = _check(same, np.full((1, 4), -3.0, dtype=np.float32), 8)
    assert list(got[1][0][:4]) == [0, 1, 2, 3] or dtype == "bf16"


def test_a_bad_row_index_has_no_candidates():
    x = _logits(4, 1000, "f32", 8)
    rows = np.array([[0, 4, 2, -1]])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _run(x, _scores(1, 4, 8), 8, rows=rows, err=err)
    assert int(err.item()) == gdn.GDN_DEVERR_BAD_INDEX
    assert set(got[1][0]) <= {0, 2}


# ------------------------------------------------------------------------------------------------
# reorder
# ------------------------------------------------------------------------------------------------
def _pools(num_slots, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(num_slots, *s, generator=g, device="cuda")
    wide = torch.randint(0, 255, (num_slots, 40), dtype=torch.uint8, generator=g, device="cuda")
    return [n(4, 16, 16), n(3 * 70, 3).to(torch.bfloat16), n(5001), wide[:, 3:10],
            torch.arange(num_slots, dtype=torch.int32, device="cuda"), n(70001).to(torch.bfloat16), n(2, 8, 128)[:, 1]]


@pytest.mark.parametrize("batch,beams", [(1, 1), (1, 4), (3, 5), (7, 32), (200, 16)])
def test_reorder(batch, beams):
    r = np.random.default_rng(batch * 100 + beams)
    num_slots = batch * beams + 2
    slots = (r.permutation(num_slots)[:batch * beams]).reshape(batch, beams).astype(np.int32)
    for parents in (np.minimum((r.random((batch, beams)) ** 2 * beams).astype(np.int32), beams - 1),
                    np.zeros((batch, beams), dtype=np.int32),                          # all from one
                    np.tile(np.arange(beams, dtype=np.int32), (batch, 1)),             # nothing to do
                    r.integers(-1, beams + 1, size=(batch, beams)).astype(np.int32)):  # some without a parent
        pools = _pools(num_slots, beams)
        want_slots, copies = ref.reorder(slots, parents)
        want = [p.clone() for p in pools]
        for w, p in zip(want, pools):
            for a, b in copies:
                w[b] = p[a]
        new = torch.full((batch, beams), -9, dtype=torch.int32, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        gdn.gdn_beam_reorder(pools, torch.from_numpy(slots).cuda(), torch.from_numpy(parents).cuda(), new, err_flags=err)
        torch.cuda.synchronize()
        np.testing.assert_array_equal(new.cpu().numpy(), want_slots)
        for w, p in zip(want, pools):
            assert torch.equal(w, p)
        assert int(err.item()) == 0


def test_reorder_more_beams_than_one_launch():
    batch, beams = 300, 8
    r = np.random.default_rng(1)
    slots = r.permutation(batch * beams).reshape(batch, beams).astype(np.int32)
    parents = r.integers(0, beams, size=(batch, beams)).astype(np.int32)
    pool = torch.randn(batch * beams, 100, device="cuda")
    want_slots, copies = ref.reorder(slots, parents)
    want = pool.clone()
    for a, b in copies:
        want[b] = pool[a]
    new = torch.empty(batch, beams, dtype=torch.int32, device="cuda")
    gdn.gdn_beam_reorder([pool], torch.from_numpy(slots).cuda(), torch.from_numpy(parents).cuda(), new)
    np.testing.assert_array_equal(new.cpu().numpy(), want_slots)
    assert torch.equal(pool, want)


def test_reorder_bad_slots_copy_nothing():
    pool = torch.randn(6, 64, device="cuda")
    before = pool.clone()
    slots = torch.tensor([[0, 9, 2], [3, 4, -1]], dtype=torch.int32, device="cuda")
    parents = torch.tensor([[0, 0, 2], [2, 2, 0]], dtype=torch.int32, device="cuda")
    new, err = torch.empty_like(slots), torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_beam_reorder([pool], slots, parents, new, err_flags=err)
    assert torch.equal(pool, before) and int(err.item()) == gdn.GDN_DEVERR_BAD_INDEX
    assert new.tolist() == [[0, 9, 2], [-1, 4, 3]]


def test_no_pools_only_maps():
    slots = torch.tensor([[5, 6]], dtype=torch.int32, device="cuda")
    new = torch.empty_like(slots)
    gdn.gdn_beam_reorder([], slots, torch.tensor([[1, 1]], dtype=torch.int32, device="cuda"), new)
    assert new.tolist() == [[6, 5]]


def test_search_step_in_a_graph():
    """Selection and reordering captured together, replayed on new logits."""
    batch, beams, V = 2, 4, 3000
    logits = _logits(8, V, "bf16", 1)
    scores = torch.from_numpy(_scores(batch, beams, 1)).cuda()
    out = torch.empty(batch, beams, device="cuda"), torch.empty(batch, beams, dtype=torch.int32, device="cuda"), \
        torch.empty(batch, beams, dtype=torch.int32, device="cuda")
    slots = torch.arange(8, dtype=torch.int32, device="cuda").view(batch, beams)
    new, pool = torch.empty_like(slots), torch.randn(8, 5000, device="cuda")
    ws = gdn.beam_select_workspace(batch, beams, V, beams)
    def step():
        gdn.gdn_beam_select(logits, scores, *out, workspace=ws)
        gdn.gdn_beam_reorder([pool], slots, out[1], new)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (2, 3):
        logits.copy_(_logits(8, V, "bf16", seed))
        before = pool.clone()
        graph.replay()
        torch.cuda.synchronize()
        _, p, t, _ = ref.select(logits.float().cpu().numpy().astype(np.float64), scores.cpu().numpy().astype(np.float64), beams)
        np.testing.assert_array_equal(out[1].cpu().numpy(), p)
        np.testing.assert_array_equal(out[2].cpu().numpy(), t)
        want, copies = ref.reorder(slots.cpu().numpy(), p)
        np.testing.assert_array_equal(new.cpu().numpy(), want)
        for a, b in copies:
            assert torch.equal(pool[b], before[a])
