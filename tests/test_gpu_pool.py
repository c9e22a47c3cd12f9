"""The operators on a pool of states against 64 bits (pool_reference), on the GPU."""
import pytest
import torch

import gated_delta_rule_85_amd as gdr
import pool_reference as ref
from gated_delta_rule_85_amd import _lib

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
I32 = dict(dtype=torch.int32)
# dtype, output, Hq, Hv, K, V
KINDS = [(BF, BF, 2, 4, 128, 128), (BF, F32, 1, 3, 128, 64), (F32, F32, 2, 2, 64, 128), (F32, BF, 3, 6, 64, 64),
         (BF, F32, 2, 4, 64, 64), (F32, F32, 1, 2, 128, 128), (BF, BF, 1, 1, 64, 128), (BF, F32, 2, 4, 128, 128)]


def say(*a):
    print(*a, flush=True)


def untouched(states, before, slots):
    """The pool's other slots hold what they held, to the bit."""
    rest = [s for s in range(before.shape[0]) if s not in slots]
    assert torch.equal(states[rest].cpu(), before[rest])


def run_recurrent(d, **kw):
    return gdr.recurrent_gated_delta_rule(d["q"], d["k"], d["v"], d["g"], d["beta"], d["states"], cu_seqlens=d["cu"],
                                          slots=d["slots"], **kw)


def run_tree(d, **kw):
    return gdr.tree_gated_delta_rule(d["q"], d["k"], d["v"], d["g"], d["beta"], d["parents"], d["states"],
                                     cu_seqlens=d["cu"], slots=d["slots"], **kw)


def run_accept(d):
    return gdr.tree_gated_delta_rule_accept(d["k"], d["v"], d["g"], d["beta"], d["parents"], d["accepted"], d["states"],
                                            cu_seqlens=d["cu"], slots=d["slots"])


# ---------------------------------------------------------------- recurrent
@pytest.mark.parametrize("dtype,out,Hq,Hv,K,V", KINDS)
@pytest.mark.parametrize("N,T,lens", [(1, 1, None), (5, 1, None), (3, 2, None), (2, 9, None), (0, 0, [1, 0, 3, 1, 7])])
def test_recurrent(dtype, out, Hq, Hv, K, V, N, T, lens):
    say("recurrent", dtype, out, Hq, Hv, K, V, N, T, lens)
    x = ref.make(N, T, Hq, Hv, K, V, dtype, lens, seed=3)
    o_want, s_want, X = ref.recurrent(x)
    d = ref.cuda(x)
    o = run_recurrent(d, output_dtype=out)
    n = T if lens is None else max(lens)
    ref.near(o, o_want, n, K, X, "o")
    ref.near(d["states"], s_want, n, K, X, "states")
    untouched(d["states"], x["states"], x["slots"].tolist())


def test_recurrent_is_the_chunked_operator_on_long_sequences():
    x = ref.make(2, 300, 2, 4, 128, 128, BF, seed=4)
    d = ref.cuda(x)
    h0 = d["states"][d["slots"].long()]
    o, ht = gdr.chunk_gated_delta_rule(d["q"], d["k"], d["v"], d["g"], d["beta"], initial_state=h0,
                                       output_final_state=True)
    o2 = run_recurrent(d)
    # the chunked operator's own parity bar is 2e-2 of the rms; it measures 1e-4 to 2.5e-4
    for a, b in ((o, o2), (ht, d["states"][d["slots"].long()])):
        assert float((a - b).abs().max()) <= 1e-3 * float(b.square().mean().sqrt())


def test_recurrent_without_slots_and_with_a_scale():
    x = ref.make(3, 2, 1, 2, 64, 64, F32, seed=5)
    x["slots"] = torch.arange(3, **I32)
    o_want, s_want, X = ref.recurrent(x, scale=0.75)
    d = ref.cuda(x)
    d["slots"] = None
    ref.near(run_recurrent(d, scale=0.75), o_want, 2, 64, X)
    ref.near(d["states"], s_want, 2, 64, X)


def test_indices_on_the_host_are_taken():
    x = ref.make(0, 0, 1, 2, 64, 64, F32, [2, 1], seed=5)
    o_want, s_want, X = ref.recurrent(x)
    d = ref.cuda(x)
    d["slots"], d["cu"] = x["slots"], x["cu"]
    ref.near(run_recurrent(d), o_want, 2, 64, X)
    ref.near(d["states"], s_want, 2, 64, X)


@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_recurrent_reads_slices_of_a_projection(T, dtype):
    """q, k, v as parts of one row, of odd batch and row strides, and one part that has to be copied."""
    x = ref.make(4, T, 2, 4, 64, 64, dtype, seed=6)
    o_want, s_want, X = ref.recurrent(x)
    d = ref.cuda(x)
    parts = [d[n].flatten(2) for n in ("q", "k", "v")]
    for pad, copied in ((8, False), (3, True)):
        row = torch.cat(parts + [torch.zeros(4, T, pad, dtype=dtype, device="cuda")], dim=-1)
        wide = torch.zeros(4, T + 2, row.shape[-1], dtype=dtype, device="cuda")
        wide[:, :T] = row
        e = dict(d, states=d["states"].clone())
        e["q"], e["k"] = wide[:, :T, :128].view(4, T, 2, 64), wide[:, :T, 128:256].view(4, T, 2, 64)
        e["v"] = wide[:, :T, 256:512].view(4, T, 4, 64)
        o = run_recurrent(e)
        ref.near(o, o_want, T, 64, X, "o %s" % copied)
        ref.near(e["states"], s_want, T, 64, X, "states %s" % copied)


@pytest.mark.parametrize("n", [5, 16, 37, 64])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("packed", [False, True])
def test_trees_read_slices_of_a_projection(n, dtype, packed):
    """Rows a projection's width apart, with NaN between the parts and behind the trees."""
    Hq, Hv, K, V = 2, 4, 64, 128
    x = ref.make(0, 0, Hq, Hv, K, V, dtype, [n, 3], seed=n) if packed else ref.make(2, n, Hq, Hv, K, V, dtype, seed=n)
    gen = torch.Generator().manual_seed(n)
    lens = [n, 3] if packed else [n, n]
    x["parents"] = torch.tensor(sum((shape_of("random", m, gen) for m in lens), []), **I32).view(x["k"].shape[:2])
    x["accepted"] = torch.tensor([n - 1, 2], **I32)
    o_want, X = ref.tree(x, x["parents"])
    s_want, X2 = ref.accept(x, x["parents"], x["accepted"])
    d = ref.cuda(x)
    B, T = x["k"].shape[:2]
    wide = torch.full((B, T + 3, 3 * 128 + 512 + 40), float("nan"), dtype=dtype, device="cuda")
    wide[:, :T, :128], wide[:, :T, 136:264], wide[:, :T, 272:784] = (d[m].flatten(2) for m in ("q", "k", "v"))
    d["q"], d["k"] = wide[:, :T, :128].view(B, T, Hq, K), wide[:, :T, 136:264].view(B, T, Hq, K)
    d["v"] = wide[:, :T, 272:784].view(B, T, Hv, V)
    assert not d["k"].is_contiguous()
    ref.near(run_tree(d), o_want, n, K, X)
    run_accept(d)
    ref.near(d["states"], s_want, n, K, X2)


def test_expanded_inputs_are_read_in_place():
    """One row for every token, and for every sequence: strides of zero."""
    x = ref.make(3, 21, 1, 2, 128, 64, BF, seed=15)
    for name in ("q", "k", "v"):
        x[name] = x[name][:1, :1].expand_as(x[name])
    x["parents"], x["accepted"] = torch.tensor([list(range(-1, 20))] * 3, **I32), torch.tensor([20] * 3, **I32)
    o_want, s_want, X = ref.recurrent(x)
    d = ref.cuda(x)
    for name in ("q", "k", "v"):
        d[name] = d[name][:1, :1].contiguous().expand_as(d[name])
    ref.near(run_tree(d), o_want, 21, 128, X)
    e = dict(d, states=d["states"].clone())
    run_accept(e)
    ref.near(run_recurrent(d), o_want, 21, 128, X)
    ref.near(d["states"], s_want, 21, 128, X)
    assert torch.equal(d["states"], e["states"])


def test_calls_from_two_threads():
    """The binding releases the interpreter's lock: two threads, a stream and a pool each."""
    import threading
    xs = [ref.make(3, 4, 2, 4, 64, 64, BF, seed=s) for s in (31, 32)]
    ds, failed = [ref.cuda(x) for x in xs], []
    torch.cuda.synchronize()

    def work(d):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(50):
                    state = d["states"].clone()
                    d["o"] = run_recurrent(dict(d, states=state))
                    d["after"] = state
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(d,)) for d in ds]
    for th in threads:
        th.start()
    for th in threads:
        th.join(60)
    assert not failed
    for x, d in zip(xs, ds):
        o_want, s_want, X = ref.recurrent(x)
        ref.near(d["o"], o_want, 4, 64, X)
        ref.near(d["after"], s_want, 4, 64, X)


def test_recurrent_on_a_pool_with_other_things_between_its_slots():
    x = ref.make(3, 1, 2, 4, 64, 64, BF, seed=7)
    o_want, s_want, X = ref.recurrent(x)
    d = ref.cuda(x)
    wide = torch.full((5, 4 * 64 * 64 + 12), 7.0, device="cuda")
    pool = wide[:, 8:8 + 4 * 64 * 64].view(5, 4, 64, 64)
    pool.copy_(d["states"])
    d["states"] = pool
    ref.near(run_recurrent(d), o_want, 1, 64, X)
    ref.near(d["states"].clone(), s_want, 1, 64, X)
    assert bool((wide[:, :8] == 7).all()) and bool((wide[:, -4:] == 7).all())


def test_padding_and_repeated_slots_are_skipped():
    """Slots of -1 and past the pool, and a slot that an earlier sequence has: zero rows, no state touched."""
    x = ref.make(0, 0, 1, 2, 64, 64, F32, [2, 1, 0, 3, 1, 1], seed=8)
    for n in ("q", "k", "v", "g", "beta"):
        x[n][:, 2] = float("nan")  # of the skipped sequence 1
    d = ref.cuda(x)
    # sequence 2 is empty and owns nothing, so that sequence 3 has slot 4; 4 repeats 0's
    d["slots"] = torch.tensor([5, -1, 4, 4, 5, 1000], **I32, device="cuda")
    o = run_recurrent(d)
    y = dict(x, q=x["q"][:, [0, 1, 3, 4, 5]], k=x["k"][:, [0, 1, 3, 4, 5]], v=x["v"][:, [0, 1, 3, 4, 5]],
             g=x["g"][:, [0, 1, 3, 4, 5]], beta=x["beta"][:, [0, 1, 3, 4, 5]], cu=torch.tensor([0, 2, 5]),
             slots=torch.tensor([5, 4]))
    o_want, s_want, X = ref.recurrent(y)
    ref.near(o[:, [0, 1, 3, 4, 5]], o_want, 3, 64, X)
    assert bool((o[:, [2, 6, 7]] == 0).all())
    ref.near(d["states"], s_want, 3, 64, X)
    untouched(d["states"], x["states"], [4, 5])


@pytest.mark.parametrize("N", [300, 1500])
def test_many_sequences_with_a_repeated_slot(N):
    """The lookup of earlier owners over more sequences than a wave has lanes, and over more
    than a wave looks through alone."""
    x = ref.make(N, 1, 1, 1, 64, 64, F32, seed=9)
    d = ref.cuda(x)
    again = {257: 3, N - 1: 130, N // 2: 0}
    slots = x["slots"].clone()
    for late, early in again.items():
        slots[late] = slots[early]
    d["slots"] = slots.cuda()
    o = run_recurrent(d)
    keep = [i for i in range(N) if i not in again]
    o_want, s_want, X = ref.recurrent(x)
    ref.near(o[keep], o_want[keep], 1, 64, X)
    assert bool((o[list(again)] == 0).all())
    lost = [int(x["slots"][i]) for i in again]
    rest = [s for s in range(N + 2) if s not in lost]
    ref.near(d["states"][rest], s_want[rest], 1, 64, X)
    assert torch.equal(d["states"][lost].cpu(), x["states"][lost])


def test_rows_behind_the_last_sequence_are_left():
    x = ref.make(0, 0, 1, 2, 64, 64, F32, [2, 1, 2], seed=10)
    x["cu"] = torch.tensor([0, 2, 3, 3], **I32)
    x["parents"] = torch.tensor([[-1, 0, -1, 0, 0]], **I32)
    for run in (run_recurrent, run_tree):
        d = ref.cuda(x)
        out = torch.full((1, 5, 2, 64), 9.0, device="cuda")
        assert run(d, out=out) is out
        assert bool((out[:, 3:] == 9).all()) and bool((out[:, :3] != 9).all())


@pytest.mark.parametrize("n", [1, 3, 17, 33, 49, 63, 64])
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_rows_behind_a_tree_are_left(n, out_dtype):
    """The tiles of 16 nodes end inside the rows: what follows belongs to nobody."""
    x = ref.make(0, 0, 2, 4, 64, 128, BF, [n, 80 - n], seed=n)
    x["parents"] = torch.tensor([list(range(-1, n - 1)) + [-1] * (80 - n)], **I32)
    for name in ("q", "k", "v", "g", "beta"):
        x[name][:, n:] = float("nan")
    first = {m: x[m][:, :n] for m in ("q", "k", "v", "g", "beta")}
    o_want, _, X = ref.recurrent(dict(x, **first, cu=torch.tensor([0, n])))
    d = ref.cuda(x)
    out = torch.full((1, 80, 4, 128), 9.0, dtype=out_dtype, device="cuda")
    run_tree(dict(d, cu=torch.tensor([0, n], **I32, device="cuda"), slots=d["slots"][:1]), out=out)
    ref.near(out[:, :n], o_want, n, 64, X)
    assert bool((out[:, n:] == 9).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tensors_that_are_not_aligned_are_copied(dtype):
    x = ref.make(2, 3, 2, 4, 64, 64, dtype, seed=14)
    x["parents"], x["accepted"] = torch.tensor([[-1, 0, 1]] * 2, **I32), torch.tensor([2, 2], **I32)
    o_want, s_want, X = ref.recurrent(x)
    for name in ("q", "k", "v"):
        d = ref.cuda(x)
        off = torch.zeros(d[name].numel() + 1, dtype=dtype, device="cuda")[1:].view(d[name].shape)
        d[name] = off.copy_(d[name])
        assert d[name].data_ptr() % 16
        ref.near(run_tree(d), o_want, 3, 64, X)
        e = dict(d, states=d["states"].clone())
        run_accept(e)
        ref.near(run_recurrent(d), o_want, 3, 64, X)
        ref.near(d["states"], s_want, 3, 64, X)
        assert torch.equal(d["states"], e["states"])


def test_offsets_out_of_range_on_the_device_touch_nothing_else():
    x = ref.make(0, 0, 1, 2, 64, 64, F32, [2, 1, 2], seed=10)
    x["parents"] = torch.tensor([[-1, 0, -1, 0, 0]], **I32)
    x["accepted"] = torch.tensor([9, 0, -7], **I32)
    for cu in ([-5, 2, 900, 4], [4, 1, 1, 3], [2 ** 31 - 1, -2 ** 31, 7, 7]):
        for run in (run_recurrent, run_tree, run_accept):
            d = ref.cuda(x)
            d["cu"] = torch.tensor(cu, **I32, device="cuda")
            guard = torch.full((12, 2, 64), 5.0, device="cuda")
            if run is run_accept:
                run(d)
            else:
                run(d, out=guard[4:9].view(1, 5, 2, 64))
            torch.cuda.synchronize()
            assert bool((guard[:4] == 5).all()) and bool((guard[9:] == 5).all())
            untouched(d["states"], x["states"], x["slots"].tolist())


def test_out_is_checked():
    d = ref.cuda(ref.make(2, 1, 1, 2, 64, 64, F32, seed=1))
    for out in (torch.empty(2, 1, 2, 65, device="cuda"), torch.empty(2, 1, 2, 64, device="cuda").half(),
                torch.empty(2, 1, 64, 2, device="cuda").mT, torch.empty(2, 1, 2, 64), d["v"],
                d["states"].view(-1)[:256].view(2, 1, 2, 64)):
        with pytest.raises(ValueError):
            run_recurrent(d, out=out)


def test_empty_batches():
    x = ref.make(2, 1, 1, 2, 64, 64, F32, seed=1)
    for y in (dict(x, **{n: x[n][:0] for n in ("q", "k", "v", "g", "beta", "slots")}),
              dict(x, **{n: x[n][:, :0] for n in ("q", "k", "v", "g", "beta")}),
              dict(x, **{n: x[n][:1, :0] for n in ("q", "k", "v", "g", "beta")}, cu=torch.tensor([0, 0, 0], **I32)),
              dict(x, **{n: x[n][:1, :0] for n in ("q", "k", "v", "g", "beta")}, cu=torch.tensor([0], **I32),
                   slots=x["slots"][:0])):
        B, T = y["q"].shape[:2]
        y["parents"] = torch.zeros(B, T, **I32)
        y["accepted"] = torch.zeros(len(y["slots"]), **I32) - 1
        d = ref.cuda(y)
        assert run_recurrent(d).shape == y["v"].shape and run_tree(d).shape == y["v"].shape
        run_accept(d)
        assert torch.equal(d["states"].cpu(), x["states"])


def test_gates_that_forget_everything():
    """g = -inf and far below any exponent: the state is cleared, and later nodes are exact."""
    x = ref.make(2, 6, 1, 2, 128, 64, F32, seed=12)
    x["g"][0, 2] = float("-inf")
    x["g"][1, 1] = -3e5
    x["g"][1, 4] = -1e30
    x["parents"] = torch.tensor([[-1, 0, 1, 2, 3, 3], [-1, 0, 1, 2, 3, 1]], **I32)
    x["accepted"] = torch.tensor([4, 5], **I32)
    o_want, s_want, X = ref.recurrent(x)
    d = ref.cuda(x)
    ref.near(run_recurrent(d), o_want, 6, 128, X)
    ref.near(d["states"], s_want, 6, 128, X)
    d = ref.cuda(x)
    o_want, X = ref.tree(x, x["parents"])
    ref.near(run_tree(d), o_want, 6, 128, X)
    run_accept(d)
    s_want, X = ref.accept(x, x["parents"], x["accepted"])
    ref.near(d["states"], s_want, 6, 128, X)


def test_offsets_past_32_bits():
    """Slots at the far end of a pool of more than 2^31 values."""
    Hv, K, V, n = 32, 128, 128, 4100
    pool = torch.empty(n, Hv, K, V, device="cuda")
    x = ref.make(2, 3, 2, Hv, K, V, BF, seed=13)
    x["parents"], x["accepted"] = torch.tensor([[-1, 0, 0], [-1, -1, 1]], **I32), torch.tensor([2, 2], **I32)
    small = dict(x, slots=torch.tensor([0, 1]), states=x["states"][:2])
    d = ref.cuda(x)
    d["states"], d["slots"] = pool, torch.tensor([n - 1, n - 3], **I32, device="cuda")
    far = [n - 1, n - 3]
    for run, want in ((run_recurrent, lambda: ref.recurrent(small)), (run_tree, lambda: ref.tree(small, x["parents"])),
                      (run_accept, lambda: ref.accept(small, x["parents"], x["accepted"]))):
        pool[far] = small["states"].cuda()
        got = run(d)
        w = want()
        if run is not run_accept:
            ref.near(got, w[0], 3, K, w[-1])
        if run is not run_tree:
            ref.near(pool[far], w[-2], 3, K, w[-1])
    pool[far] = small["states"].cuda()
    pool[:4] = 1.0
    gdr.copy_states(pool, torch.tensor([0, n - 3, n - 1], **I32, device="cuda"),
                    torch.tensor([n - 3, n - 1, 2], **I32, device="cuda"))
    assert torch.equal(pool[0].cpu(), small["states"][1]) and torch.equal(pool[n - 3].cpu(), small["states"][0])
    assert bool((pool[n - 1] == 1).all())


# ---------------------------------------------------------------- trees
def shape_of(kind, n, gen):
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] + [0] * (n - 1)
    if kind == "roots":
        return [-1] * n
    if kind == "binary":
        return [(i - 1) // 2 if i else -1 for i in range(n)]
    return [int(torch.randint(-1, i, (1,), generator=gen)) if i else -1 for i in range(n)]


@pytest.mark.parametrize("dtype,out,Hq,Hv,K,V", KINDS)
@pytest.mark.parametrize("n", [1, 2, 7, 15, 16, 17, 32, 33, 47, 48, 49, 63, 64])
def test_tree(dtype, out, Hq, Hv, K, V, n):
    gen = torch.Generator().manual_seed(n)
    kinds = ["random", ["chain", "star", "roots", "binary"][n % 4]]
    say("tree", dtype, out, Hq, Hv, K, V, n, kinds)
    x = ref.make(2, n, Hq, Hv, K, V, dtype, seed=n)
    x["parents"] = torch.tensor([shape_of(k, n, gen) for k in kinds], **I32)
    o_want, X = ref.tree(x, x["parents"])
    d = ref.cuda(x)
    o = run_tree(d, output_dtype=out)
    assert torch.equal(d["states"].cpu(), x["states"])
    ref.near(o, o_want, n, K, X, "o")


@pytest.mark.parametrize("kind", ["chain", "star", "roots", "binary", "random"])
def test_tree_shapes(kind):
    gen = torch.Generator().manual_seed(1)
    x = ref.make(3, 64, 1, 2, 128, 128, BF, seed=2)
    x["parents"] = torch.tensor([shape_of(kind, 64, gen) for _ in range(3)], **I32)
    o_want, X = ref.tree(x, x["parents"])
    ref.near(run_tree(ref.cuda(x)), o_want, 64, 128, X)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_packed_trees(dtype):
    lens = [5, 0, 64, 1, 17, 33, 48]
    gen = torch.Generator().manual_seed(3)
    x = ref.make(0, 0, 2, 4, 128, 64, dtype, lens, seed=3)
    x["parents"] = torch.tensor([sum((shape_of("random", n, gen) for n in lens), [])], **I32)
    x["accepted"] = torch.tensor([4, -1, 63, 0, 11, 30, -1], **I32)
    o_want, X = ref.tree(x, x["parents"])
    d = ref.cuda(x)
    ref.near(run_tree(d), o_want, 64, 128, X)
    run_accept(d)
    s_want, X = ref.accept(x, x["parents"], x["accepted"])
    ref.near(d["states"], s_want, 64, 128, X)
    untouched(d["states"], x["states"], [int(s) for s, n in zip(x["slots"], x["accepted"]) if n >= 0])


def test_a_chain_is_the_recurrent_form_and_trees_may_share_a_slot():
    x = ref.make(1, 8, 2, 4, 128, 128, BF, seed=4)
    d = ref.cuda(x)
    d["parents"] = torch.tensor([[-1, 0, 1, 2, 3, 4, 5, 6]], **I32, device="cuda")
    two = {n: torch.cat([d[n], d[n]]) for n in ("q", "k", "v", "g", "beta", "parents", "slots")}
    o = run_tree(dict(d, **two))
    assert torch.equal(o[0], o[1])
    want, _, X = ref.recurrent(x)
    ref.near(o[:1], want, 8, 128, X)


@pytest.mark.parametrize("dtype,out", [(BF, F32), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("n", [14, 50])
@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nonfinite_nodes_reach_their_descendants_only(dtype, out, n, name, value):
    """Siblings and ancestors of a node with NaN or an infinity (a g of -inf is legal) are as without it."""
    x = ref.make(1, n, 1, 2, 128, 128, dtype, seed=5)
    parents = shape_of("random", n, torch.Generator().manual_seed(n))
    x["parents"] = torch.tensor([parents], **I32)
    o_want, X = ref.tree(x, x["parents"])
    bad, col = n // 3, 37
    y = dict(x)
    y[name] = x[name].clone()
    if name in ("g", "beta"):
        y[name][0, bad, 0] = value
    else:
        y[name][0, bad, 0, col] = value
    o = run_tree(ref.cuda(y), output_dtype=out)
    hit = [i for i in range(n) if (i == bad if name == "q" else bad in ref.path_of(parents, i))]
    fine = [i for i in range(n) if i not in hit]
    assert fine and hit
    # head 1 shares q and k with head 0, but not v, g and beta
    heads = [0, 1] if name in ("q", "k") else [0]
    cols = [col] if name == "v" else list(range(128))
    ok = torch.ones(1, n, 2, 128, dtype=torch.bool)
    for i in hit:
        for h in heads:
            ok[0, i, h, cols] = False
    got = o.cpu()
    assert not bool(torch.isfinite(got[~ok]).any())
    ref.near(torch.where(ok, got, 0), torch.where(ok, o_want, 0.0), n, 128, X)


def test_parents_that_are_no_earlier_nodes_count_as_none():
    x = ref.make(1, 5, 1, 1, 64, 64, F32, seed=6)
    x["parents"] = torch.tensor([[-1, 0, -1, -1, 2]], **I32)
    o_want, X = ref.tree(x, x["parents"])
    x["accepted"] = torch.tensor([3], **I32)
    s_want, X2 = ref.accept(x, x["parents"], x["accepted"])
    d = ref.cuda(x)
    d["parents"] = torch.tensor([[0, 0, 2, 64, 2]], **I32, device="cuda")
    ref.near(run_tree(d), o_want, 5, 64, X)
    run_accept(d)
    ref.near(d["states"], s_want, 5, 64, X2)


def test_trees_without_a_slot_or_of_too_many_nodes():
    x = ref.make(0, 0, 1, 2, 64, 64, BF, [3, 65, 64], seed=7)
    x["parents"] = torch.full((1, 132), -1, **I32)
    d = ref.cuda(x)
    d["slots"] = torch.tensor([-1, 0, 1], **I32, device="cuda")
    d["accepted"] = torch.tensor([2, 64, 63], **I32, device="cuda")
    o = run_tree(d)
    assert bool((o[:, :3] == 0).all()) and bool(torch.isnan(o[:, 3:68]).all()) and bool(torch.isfinite(o[:, 68:]).all())
    run_accept(d)
    untouched(d["states"], x["states"], [1])
    assert not torch.equal(d["states"][1].cpu(), x["states"][1])


# ---------------------------------------------------------------- acceptance
@pytest.mark.parametrize("dtype,out,Hq,Hv,K,V", KINDS)
def test_accept_is_decoding_the_path(dtype, out, Hq, Hv, K, V):
    """Against 64 bits, and to the bit against the recurrent form on the path's tokens."""
    n = 21
    gen = torch.Generator().manual_seed(2)
    parents = [shape_of(k, n, gen) for k in ("random", "chain", "binary", "star")]
    x = ref.make(4, n, Hq, Hv, K, V, dtype, seed=11)
    x["parents"], x["accepted"] = torch.tensor(parents, **I32), torch.tensor([20, 13, 17, -1], **I32)
    s_want, X = ref.accept(x, x["parents"], x["accepted"])
    d = ref.cuda(x)
    assert run_accept(d) is d["states"]
    ref.near(d["states"], s_want, n, K, X)
    untouched(d["states"], x["states"], x["slots"][:3].tolist())
    e = ref.cuda(x)
    for j in range(3):
        p = ref.path_of(parents[j], int(x["accepted"][j]))
        part = {m: e[m][j:j + 1, p] for m in ("q", "k", "v", "g", "beta")}
        run_recurrent(dict(part, states=e["states"], slots=e["slots"][j:j + 1], cu=None))
    assert torch.equal(d["states"], e["states"])


def test_accept_skips_padding_and_repeated_slots():
    x = ref.make(4, 3, 1, 2, 64, 64, F32, seed=12)
    x["parents"], x["accepted"] = torch.tensor([[-1, 0, 1]] * 4, **I32), torch.tensor([2, 1, 2, 3], **I32)
    x["slots"] = torch.tensor([5, 4, 3, 0], **I32)
    s_want, X = ref.accept(x, x["parents"], torch.tensor([2, 1, -1, -1]))
    d = ref.cuda(x)
    d["slots"] = torch.tensor([5, 4, 5, 0], **I32, device="cuda")  # the third repeats; the fourth accepts no node
    run_accept(d)
    ref.near(d["states"], s_want, 3, 64, X)
    untouched(d["states"], x["states"], [4, 5])


# ---------------------------------------------------------------- copies
def copied(states, dst, src, source=None):
    before, after = (states if source is None else source).clone(), states.clone()
    for a, b in zip(dst.tolist(), src.tolist()):
        if 0 <= a < states.shape[-4] and b < before.shape[-4]:
            after[..., a, :, :, :] = before[..., b, :, :, :] if b >= 0 else 0.0
    return after


@pytest.mark.parametrize("n", [0, 1, 2, 3, 4, 5, 16, 17, 64, 65, 200, 256, 257, 1024, 1025, 4096])
def test_copies_of_any_number(n):
    say("copy", n)
    gen = torch.Generator().manual_seed(n)
    slots = max(4, n + 3)
    states = torch.randn(slots, 1, 64, 64, generator=gen)
    dst = torch.randperm(slots, generator=gen)[:n].to(torch.int32)
    src = torch.randint(-1, slots, (n,), generator=gen, dtype=torch.int32)
    want = copied(states, dst, src)
    pool = states.cuda()
    assert gdr.copy_states(pool, dst.cuda(), src.cuda()) is pool
    assert torch.equal(pool.cpu(), want)


@pytest.mark.parametrize("Hv,K,V", [(1, 64, 64), (3, 128, 64), (5, 64, 64), (32, 128, 128)])
def test_permutations_forks_and_clears(Hv, K, V):
    states = torch.randn(9, Hv, K, V, generator=torch.Generator().manual_seed(1))
    for dst, src in (([1, 2, 3, 0], [0, 1, 2, 3]), ([8, 7], [7, 8]), ([0, 1, 2, 3, 4, 5, 6, 7, 8], [4] * 9),
                     ([3, 2, 1], [2, 1, -1]), ([5], [5]), ([0, 1, 2, 3, 4, 5, 6, 7, 8], [-1] * 9)):
        dst, src = torch.tensor(dst, **I32), torch.tensor(src, **I32)
        pool = states.cuda()
        gdr.copy_states(pool, dst, src.cuda())  # dst on the host
        assert torch.equal(pool.cpu(), copied(states, dst, src)), (dst, src)


@pytest.mark.parametrize("n", [6, 40, 300, 1500])
def test_the_last_of_equal_destinations_stands_and_bad_entries_are_skipped(n):
    gen = torch.Generator().manual_seed(n)
    states = torch.randn(n, 2, 64, 64, generator=gen)
    dst = torch.randint(-3, n // 2, (n,), generator=gen, dtype=torch.int32)
    src = torch.randint(-2, n + 4, (n,), generator=gen, dtype=torch.int32)
    dst[n // 2], src[n // 3] = 2 ** 31 - 1, 2 ** 31 - 1
    dst[1], src[1] = -2 ** 31, 0
    for _ in range(2):
        pool = states.cuda()
        gdr.copy_states(pool, dst.cuda(), src.cuda())
        assert torch.equal(pool.cpu(), copied(states, dst, src))


@pytest.mark.parametrize("slots_first", [False, True])
def test_copies_in_every_layer(slots_first):
    states = torch.randn(3, 7, 2, 64, 128, generator=torch.Generator().manual_seed(2))
    dst, src = torch.tensor([0, 3, 6, 1], **I32), torch.tensor([3, 0, -1, 0], **I32)
    pool = states.transpose(0, 1).contiguous().cuda().transpose(0, 1) if slots_first else states.cuda()
    gdr.copy_states(pool, dst.cuda(), src.cuda())
    assert torch.equal(pool.cpu(), copied(states, dst, src))
    part = (states.transpose(0, 1).contiguous().cuda().transpose(0, 1) if slots_first else states.cuda())
    gdr.copy_states(part[:, ::2], dst.clamp(max=3).cuda(), src.clamp(max=3).cuda())
    want = states.clone()
    want[:, ::2] = copied(states[:, ::2], dst.clamp(max=3), src.clamp(max=3))
    assert torch.equal(part.cpu(), want)


def test_copies_from_another_pool():
    gen = torch.Generator().manual_seed(3)
    states, source = torch.randn(5, 2, 64, 64, generator=gen), torch.randn(8, 2, 64, 64, generator=gen)
    dst, src = torch.tensor([4, 0, 2], **I32), torch.tensor([7, 7, -1], **I32)
    pool = states.cuda()
    gdr.copy_states(pool, dst.cuda(), src.cuda(), source.cuda())
    assert torch.equal(pool.cpu(), copied(states, dst, src, source))
    pool = states.cuda()
    gdr.copy_states(pool[:2], torch.tensor([0, 1], **I32), torch.tensor([1, 2], **I32), pool[2:])
    assert torch.equal(pool.cpu(), torch.cat([states[3:5], states[2:]]))


# ---------------------------------------------------------------- together
def test_serving_from_prefill_to_release():
    """Prefill, placement in the pool, decode, verification of trees, acceptance, a fork and a
    compaction, against 64 bits over the whole run."""
    Hq, Hv, K, V, N = 2, 4, 128, 128, 3
    lens = [70, 5, 129]
    x = ref.make(0, 0, Hq, Hv, K, V, BF, lens, seed=20)
    d = ref.cuda(x)
    _, final = gdr.chunk_gated_delta_rule(d["q"], d["k"], d["v"], d["g"], d["beta"], cu_seqlens=d["cu"],
                                          output_final_state=True)
    slots = torch.tensor([6, 1, 3], **I32)
    pool = torch.full((8, Hv, K, V), float("nan"), device="cuda")
    gdr.copy_states(pool, slots.cuda(), torch.arange(N, **I32, device="cuda"), final)
    zero = dict(x, states=torch.zeros(N, Hv, K, V), slots=torch.arange(N))
    _, want, X = ref.recurrent(zero)
    # the prefill's states carry its own error (two bf16 pieces per product: about 2e-5 of the
    # rms); later tokens do not enlarge it
    bar = 1e-3 * float(want.square().mean().sqrt())
    assert float((pool[slots.long()].cpu() - want).abs().max()) <= bar
    for t in range(3):
        y = ref.make(N, 1, Hq, Hv, K, V, BF, seed=21 + t)
        e = dict(ref.cuda(y), states=pool, slots=slots.cuda())
        o = run_recurrent(e)
        o_want, want, _ = ref.recurrent(dict(y, states=want, slots=torch.arange(N)))
        assert float((o.cpu() - o_want).abs().max()) <= bar
    n = 13
    y = ref.make(N, n, Hq, Hv, K, V, BF, seed=30)
    y["parents"] = torch.tensor([shape_of("random", n, torch.Generator().manual_seed(j)) for j in range(N)], **I32)
    y["accepted"] = torch.tensor([12, -1, 5], **I32)
    e = dict(ref.cuda(y), states=pool, slots=slots.cuda())
    o = run_tree(e)
    ref_in = dict(y, states=want, slots=torch.arange(N))
    o_want, _ = ref.tree(ref_in, y["parents"])
    assert float((o.cpu() - o_want).abs().max()) <= bar
    run_accept(e)
    want, _ = ref.accept(ref_in, y["parents"], y["accepted"])
    assert float((pool[slots.long()].cpu() - want).abs().max()) <= bar
    # fork sequence 0 into slots 0 and 2, release sequence 1, move sequence 2 down to its slot
    gdr.copy_states(pool, torch.tensor([0, 2, 1, 3], **I32), torch.tensor([6, 6, 3, -1], **I32))
    for s, j in ((0, 0), (2, 0), (6, 0), (1, 2)):
        assert float((pool[s].cpu() - want[j]).abs().max()) <= bar
    assert bool((pool[3] == 0).all())


def test_captured_calls_replay_as_eager_ones():
    """All four in one graph, replayed with new inputs and eager work in between."""
    N, n, Hq, Hv, K, V = 3, 9, 2, 4, 64, 128
    def fresh(seed):
        x = ref.make(N, 1, Hq, Hv, K, V, BF, seed=seed)
        t = ref.make(N, n, Hq, Hv, K, V, BF, seed=seed + 50)
        gen = torch.Generator().manual_seed(seed)
        t["parents"] = torch.tensor([shape_of("random", n, gen) for _ in range(N)], **I32)
        t["accepted"] = torch.randint(-1, n, (N,), generator=gen, dtype=torch.int32)
        t["slots"] = x["slots"]
        m = dict(dst=torch.randperm(5, generator=gen)[:4].to(torch.int32),
                 src=torch.randint(-1, 5, (4,), generator=gen, dtype=torch.int32))
        return ref.cuda(x), ref.cuda(t), ref.cuda(m)
    def go(x, t, m, o, ot):
        run_recurrent(x, out=o)
        t = dict(t, states=x["states"])
        run_tree(t, out=ot)
        run_accept(t)
        gdr.copy_states(x["states"], m["dst"], m["src"])
    x, t, m = fresh(1)
    o, ot = torch.zeros(N, 1, Hv, V, device="cuda"), torch.zeros(N, n, Hv, V, device="cuda")
    go(*fresh(7), o, ot)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(x, t, m, o, ot)
    for rep in range(3):
        say("replay", rep)
        for have, new in zip((x, t, m), fresh(10 + rep)):
            for name, v in new.items():
                if v is not None:
                    have[name].copy_(v)
        e = [{a: b.clone() if b is not None else None for a, b in s.items()} for s in (x, t, m)]
        oe, ote = torch.full_like(o, 3), torch.full_like(ot, 3)
        go(*e, oe, ote)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, oe) and torch.equal(ot, ote) and torch.equal(x["states"], e[0]["states"])
    del graph


def test_calls_on_two_streams():
    """The call's own stream is the current one, and calls on several streams do not meet."""
    xs = [ref.make(4, 2, 2, 4, 128, 128, BF, seed=s) for s in (1, 2)]
    ds = [ref.cuda(x) for x in xs]
    for x in xs:
        x["parents"] = torch.tensor([[-1, 0]] * 4, **I32)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    outs = []
    for d, s, x in zip(ds, streams, xs):
        with torch.cuda.stream(s):
            p = x["parents"].cuda()
            outs.append((run_tree(dict(d, parents=p)), run_recurrent(d)))
    torch.cuda.synchronize()
    for x, d, (ot, o) in zip(xs, ds, outs):
        o_want, s_want, X = ref.recurrent(x)
        ref.near(o, o_want, 2, 128, X)
        ref.near(ot, o_want, 2, 128, X)
        ref.near(d["states"], s_want, 2, 128, X)


@pytest.mark.parametrize("op", ["recurrent", "accept", "copy"])
def test_a_backward_that_saved_the_states_notices_that_they_changed(op):
    d = ref.cuda(ref.make(2, 3, 1, 2, 64, 64, F32, seed=3, extra_slots=0))
    d["slots"] = None
    q = d["q"].clone().requires_grad_()
    o, _ = gdr.chunk_gated_delta_rule(q, d["k"], d["v"], d["g"], d["beta"], initial_state=d["states"])
    run_tree(dict(d, parents=torch.full((2, 3), -1, **I32)))  # reads them only
    o.sum().backward(retain_graph=True)
    if op == "recurrent":
        run_recurrent(d)
    elif op == "accept":
        run_accept(dict(d, parents=torch.full((2, 3), -1, **I32), accepted=torch.tensor([0, 1], **I32)))
    else:
        gdr.copy_states(d["states"], torch.tensor([0], **I32), torch.tensor([-1], **I32))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        o.sum().backward()
    with torch.inference_mode():
        e = ref.cuda(ref.make(1, 1, 1, 2, 64, 64, F32))
        run_recurrent(e, out=torch.empty_like(e["v"]))


@pytest.mark.parametrize("n", [1, 5, 40, 300, 1100])
def test_copies_of_odd_sizes_through_the_c_abi(n):
    """Slots of any multiple of 16 bytes, unequal strides, bytes between the slots and layers left alone."""
    import ctypes
    gen = torch.Generator().manual_seed(n)
    n_dst, n_src, layers, words = n + 2, n + 5, 3, 4 * 37
    dst = torch.randint(0, 1 << 30, (layers, n_dst, words + 8), generator=gen, dtype=torch.int32)
    src = torch.randint(0, 1 << 30, (layers, n_src, words + 4), generator=gen, dtype=torch.int32)
    to = torch.randperm(n_dst, generator=gen)[:n].to(torch.int32)
    frm = torch.randint(-1, n_src, (n,), generator=gen, dtype=torch.int32)
    want = dst.clone()
    for a, b in zip(to.tolist(), frm.tolist()):
        want[:, a, :words] = src[:, b, :words] if b >= 0 else 0
    d, s, t, f = dst.cuda(), src.cuda(), to.cuda(), frm.cuda()
    a = _lib.CopyArgs(n, n_dst, n_src, 4 * words, 4 * (words + 8), 4 * (words + 4), layers, 4 * n_dst * (words + 8),
                      4 * n_src * (words + 4), t.data_ptr(), f.data_ptr(), d.data_ptr(), s.data_ptr())
    assert _lib.lib.gdr_copy_states(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(d.cpu(), want)


def test_errors_of_the_library_name_their_entry_point():
    x = ref.cuda(ref.make(1, 1, 1, 1, 96, 64, F32))
    with pytest.raises(_lib.GdrError, match="gdr_step") as e:
        run_recurrent(x)
    assert e.value.code == _lib.ENOTSUP
    x["parents"] = x["accepted"] = torch.full((1, 1), -1, **I32)
    with pytest.raises(_lib.GdrError, match="gdr_tree "):
        run_tree(x)
    with pytest.raises(_lib.GdrError, match="gdr_tree_accept"):
        run_accept(dict(x, accepted=x["accepted"][0]))


# A small difference of two values near 1, in each of a tree's products: every product and
# partial sum below is exact in fp32, so the result is the difference to the bit, which two bf16
# pieces of either operand (1, and 8 bits from 2^-10 on) would lose
BASE, TINY = 1 + 2.0 ** -10, 3 * 2.0 ** -20


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [2, 20, 64])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 128)])
def test_tree_products_keep_what_is_small_by_cancellation(dtype, out, n, K, V):
    say("cancellation", dtype, out, n, K, V)
    x = dict(q=torch.zeros(1, n, 1, K, dtype=dtype), k=torch.zeros(1, n, 1, K, dtype=dtype),
             v=torch.zeros(1, n, 1, V, dtype=dtype), g=torch.zeros(1, n, 1), beta=torch.zeros(1, n, 1),
             states=torch.zeros(1, 1, K, V), slots=torch.zeros(1, **I32), cu=None)
    x["parents"] = torch.tensor([list(range(-1, n - 1))], **I32)

    def last(**change):
        return run_tree(ref.cuda(dict(x, **change)), scale=1.0, output_dtype=out)[0, -1, 0].float().cpu()

    half = x["q"].clone()
    half[0, -1, 0, :2] = torch.tensor([0.5, -0.5])
    states = x["states"].clone()
    states[0, 0, 0], states[0, 0, 1] = BASE + TINY, BASE
    # o = q h
    assert bool((last(q=half, states=states) == TINY / 2).all())
    # o = q h + (q . k) u, u = -k h
    beta = x["beta"].clone()
    beta[0, -1] = 1
    assert bool((last(q=half, k=half, states=states, beta=beta) == TINY / 4).all())
    if dtype is F32:
        q, one = x["q"].clone(), torch.ones_like(states)
        q[0, -1, 0, :2] = torch.tensor([BASE + TINY, -BASE])
        assert bool((last(q=q, states=one) == TINY).all())
        # o = (q . k0) u0 + (q . k1) u1 of the first two nodes, in q's values and in v's (n = 2: the
        # last node is the second, whose own key is zero elsewhere)
        k, v, beta = x["k"].clone(), x["v"].clone(), x["beta"].clone()
        k[0, 0, 0, 0] = k[0, 1, 0, 1] = 1
        beta[0, :2] = 1
        v[0, :2] = 1
        assert bool((last(q=q, k=k, v=v, beta=beta) == TINY).all())
        v[0, 0], v[0, 1] = BASE + TINY, BASE
        assert bool((last(q=half, k=k, v=v, beta=beta) == TINY / 2).all())


@pytest.mark.parametrize("dtype,out", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("n,at", [(6, 0), (14, 7), (50, 34), (50, 14), (64, 60)])
@pytest.mark.parametrize("size", [1e12, 1e15, 1e18])
@pytest.mark.parametrize("D", [64, 128])
def test_large_finite_nodes_reach_their_descendants_only(dtype, out, n, at, size, D):
    """Two large keys on one path, within a tile of 16 nodes and across two: products of their
    scores leave fp32's range where each of them, or each of the scores, does not."""
    say("large keys", dtype, out, n, at, size, D)
    x = ref.make(1, n, 1, 2, D, D, dtype, seed=6)
    parents = shape_of("random", n, torch.Generator().manual_seed(n + at))
    for i, up in ((at + 1, at), (at + 2, at + 1), (at + 3, at + 2)):
        parents[i] = up
    for i in range(at + 4, n):  # the others hang on other nodes
        if at < parents[i] < at + 4:
            parents[i] = at if i % 2 else -1
    x["parents"] = torch.tensor([parents], **I32)
    o_want, X = ref.tree(x, x["parents"])
    y = dict(x, k=x["k"].clone())
    y["k"][0, at + 1:at + 3] *= size
    o = run_tree(ref.cuda(y), output_dtype=out)
    fine = [i for i in range(n) if at + 1 not in ref.path_of(parents, i)]
    assert len(fine) == n - 3
    ref.near(o[:, fine], o_want[:, fine], n, D, X)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("n", [14, 50])
@pytest.mark.parametrize("value", [torch.finfo(F32).min, torch.finfo(F32).max, 2.0 ** 127, float(torch.finfo(BF).min)])
def test_values_at_the_ends_of_fp32_stay_in_their_column_and_path(out, n, value):
    """A value next to fp32's largest, which bfloat16 rounds to an infinity, in one column of one node:
    that column of the node and its descendants follows it, all else is as without it."""
    say("large value", out, n, value)
    x = ref.make(1, n, 1, 2, 128, 128, F32, seed=7)
    parents = shape_of("random", n, torch.Generator().manual_seed(n))
    bad, col = n // 3, 37
    parents[bad + 1], parents[bad + 2] = bad, bad - 1
    x["parents"] = torch.tensor([parents], **I32)
    x["beta"][0, bad, 0] = 1.0
    o_want, X = ref.tree(x, x["parents"])
    y = dict(x, v=x["v"].clone())
    y["v"][0, bad, 0, col] = value
    o_large, X_large = ref.tree(y, x["parents"])
    got = run_tree(ref.cuda(y), output_dtype=out)
    hit = [i for i in range(n) if bad in ref.path_of(parents, i)]
    assert 1 < len(hit) < n
    ref.near(got[:, hit, 0, col], o_large[:, hit, 0, col], n, 128, X_large)
    ok = torch.ones(1, n, 2, 128, dtype=torch.bool)
    ok[0, hit, 0, col] = False
    ref.near(torch.where(ok, got.cpu(), 0), torch.where(ok, o_want, 0.0), n, 128, X)


@pytest.mark.parametrize("layers", [0, 3])
def test_copies_between_pools_that_share_an_allocation(layers):
    """Two pools whose states lie between each other's."""
    both = torch.randn((layers or 1), 7, 2, 2, 64, 64, generator=torch.Generator().manual_seed(4))
    dst, src = torch.tensor([6, 0, 3, 1], **I32), torch.tensor([2, 6, -1, 2], **I32)
    buf = both.cuda()
    states, source = buf[:, :, 0], buf[:, :, 1]
    want = both.clone()
    want[:, :, 0] = copied(both[:, :, 0], dst, src, both[:, :, 1])
    if not layers:
        states, source = states[0], source[0]
    gdr.copy_states(states, dst.cuda(), src.cuda(), source)
    assert torch.equal(buf.cpu(), want)


def test_indices_on_the_device_are_not_waited_for():
    """A call returns while earlier work of its stream still runs."""
    x = ref.make(0, 0, 1, 2, 64, 64, F32, [2, 1], seed=5)
    x["parents"], x["accepted"] = torch.tensor([[-1, 0, -1]], **I32), torch.tensor([1, 0], **I32)
    d = ref.cuda(x)
    dst, src = torch.tensor([0], **I32, device="cuda"), torch.tensor([1], **I32, device="cuda")
    calls = (lambda: run_recurrent(d), lambda: run_tree(d), lambda: run_accept(d),
             lambda: gdr.copy_states(d["states"], dst, src))
    for call in calls:
        call()
    torch.cuda.synchronize()
    for call in calls:
        torch.cuda._sleep(100_000_000)
        before = torch.cuda.Event()
        before.record()
        call()
        assert not before.query()
        torch.cuda.synchronize()


EXTREMES = [float("nan"), float("inf"), float("-inf"), 3.3e38, -3.38e38, 1e38, 1e30, 1e20, -1e19, 1e12, 1e-40, -1e7]


@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("seed", range(12))
def test_any_values_stay_with_their_nodes_and_columns(dtype, out, seed):
    """Several nodes and a column of the state with values of any kind: what does not descend from
    them is as without them."""
    import random
    rng = random.Random(seed)
    K, V = rng.choice([64, 128]), rng.choice([64, 128])
    n = rng.choice([5, 16, 17, 31, 33, 48, 50, 64])
    say("extremes", dtype, out, seed, K, V, n)
    x = ref.make(1, n, 1, 2, K, V, dtype, seed=seed)
    parents = shape_of(rng.choice(["random", "binary", "star"]), n, torch.Generator().manual_seed(seed))
    x["parents"] = torch.tensor([parents], **I32)
    o_want, X = ref.tree(x, x["parents"])
    y = {a: b.clone() if isinstance(b, torch.Tensor) else b for a, b in x.items()}
    bad = set(rng.sample(range(1, n), max(1, n // 8)))
    extremes = EXTREMES + ([torch.finfo(F32).min] if dtype is F32 else [])
    for i in bad:
        for name in ("q", "k", "v"):
            how = rng.random()
            if how < 0.3:
                y[name][0, i] = rng.choice(extremes)
            elif how < 0.6:
                y[name][0, i, 0, rng.randrange(64)] = rng.choice(extremes)
            elif how < 0.7:
                y[name][0, i] *= rng.choice([1e10, 1e15, 1e20, 1e30])
        if rng.random() < 0.5:
            y["g"][0, i] = rng.choice(EXTREMES[:3] + [-3e38, 3e38, 88.0, 90.0, -250.0, 200.0])
        if rng.random() < 0.4:
            y["beta"][0, i] = rng.choice(EXTREMES[:3] + [1e30, -1e38, 0.0, 2.0])
    row, col = rng.randrange(K), rng.randrange(V)
    y["states"][int(x["slots"][0]), 0, row, col] = rng.choice(EXTREMES + [torch.finfo(F32).min])
    o = run_tree(ref.cuda(y), output_dtype=out).cpu()
    fine = [i for i in range(n) if not bad & set(ref.path_of(parents, i))]
    assert fine
    ok = torch.ones(1, len(fine), 2, V, dtype=torch.bool)
    ok[:, :, 0, col] = False
    ref.near(torch.where(ok, o[:, fine], 0), torch.where(ok, o_want[:, fine], 0.0), n, K, X)
