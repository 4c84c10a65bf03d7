"""The operators over sequences inside captured CUDA graphs, on other streams
and from several threads, and what they leave alone."""
import threading

import pytest
import torch

from helpers import muon

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layers():
    muon()
    from newton_schulz_05_gb300 import layers
    return layers


def inputs(b=3, t=70, v=3001, seed=0, dtype=torch.float32):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    return dict(gate=n(b, t, 192).to(dtype), x=n(b, t, 192).to(dtype), state=n(b, 192),
                starts=torch.rand(b, t, generator=gen, device="cuda") < 0.05,
                joint=n(b, t, 8, 64).to(dtype), w=n(64), logits=n(b, t, v).to(dtype),
                tokens=torch.randint(0, v, (b, t), generator=gen, device="cuda"), old=-n(b, t).abs(),
                adv=n(b, t), mask=torch.rand(b, t, generator=gen, device="cuda") < 0.8)


def chain(layers, i, table):
    """Every operator and every gradient once."""
    s = layers.gated_scan_forward(i["gate"], i["x"], state=i["state"], starts=i["starts"])
    sg = layers.gated_scan_backward(s.h, i["gate"], i["x"], s.h, state=i["state"], dstate=s.state, starts=i["starts"])
    q, k = i["joint"][:, :, :5], i["joint"][:, :, 5:7]
    h = layers.norm_rotate_heads_forward(q, k, i["w"], i["w"], cos=table[0], sin=table[1])
    hg = layers.norm_rotate_heads_backward(h.q, h.k, q, k, i["w"], i["w"], cos=table[0], sin=table[1])
    p = layers.token_log_probs_forward(i["logits"], i["tokens"], scale=0.9)
    o = layers.policy_loss_forward(p.log_probs, i["old"], i["adv"], ref_log_probs=i["old"], token_mask=i["mask"], kl=0.1)
    d = layers.policy_loss_backward(p.log_probs, i["old"], i["adv"], o.weights, dloss=o.loss, ref_log_probs=i["old"],
                                    token_mask=i["mask"], kl=0.1)
    return [*s, *sg, *h, *hg, *p, *o, d, layers.token_log_probs_backward(d, i["logits"], i["tokens"], p.lse, scale=0.9)]


def captured(layers, i, table):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain(layers, i, table)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(layers, i, table)
    return graph, got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("b,t", [(2, 1), (3, 70), (1, 2500), (40, 130)])
def test_replayed_graph_gives_the_same_bits(layers, b, t, dtype):
    table = layers.rotation_table(t, 64)
    i = inputs(b, t, v=500, dtype=dtype)
    want = [x.clone() for x in chain(layers, i, table)]
    graph, got = captured(layers, i, table)
    for _ in range(3):
        for x in got:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(got, want))


def test_two_graphs_replayed_at_once_share_nothing(layers):
    table = layers.rotation_table(2500, 64)
    sets = [inputs(2, 2500, v=300, seed=s) for s in (1, 2)]
    want = [[x.clone() for x in chain(layers, i, table)] for i in sets]
    pairs = [captured(layers, i, table) for i in sets]
    streams = [torch.cuda.Stream() for _ in pairs]
    for _ in range(5):
        for s, (graph, _) in zip(streams, pairs):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for w, (_, got) in zip(want, pairs):
            assert all(torch.equal(a, c) for a, c in zip(got, w))


def test_a_captured_training_step(layers):
    """Forward and backward through the differentiable functions under one capture, from
    leaves of its own (an eager graph of the same leaves must not be alive meanwhile)."""
    table = layers.rotation_table(50, 64)
    i = inputs(2, 50, v=200)
    leaves = [i[n].clone().requires_grad_() for n in ("gate", "x", "joint", "logits", "w")]

    def step():
        gate, x, joint, logits, w = leaves
        s = layers.gated_scan(gate, x, starts=i["starts"])
        h = layers.norm_rotate_heads(joint[:, :, :5], joint[:, :, 5:7], w, w, cos=table[0], sin=table[1])
        o = layers.policy_loss(layers.token_log_probs(logits, i["tokens"]), i["old"], i["adv"], token_mask=i["mask"])
        return torch.autograd.grad(o.loss + s.h.square().mean() + h.q.mean() + h.k.square().mean() * 0.5, leaves)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [g.clone() for g in step()]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_calls_on_a_stream_of_their_own(layers):
    table = layers.rotation_table(300, 64)
    i = inputs(4, 300)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    on = dict(stream=s)
    o = layers.gated_scan_forward(i["gate"], i["x"], state=i["state"], **on)
    g = layers.gated_scan_backward(o.h, i["gate"], i["x"], o.h, dstate=o.state, **on)
    q = i["joint"]
    h = layers.norm_rotate_heads_forward(q, q, i["w"], i["w"], cos=table[0], sin=table[1], **on)
    hg = layers.norm_rotate_heads_backward(h.q, h.k, q, q, i["w"], i["w"], cos=table[0], sin=table[1], **on)
    p = layers.token_log_probs_forward(i["logits"], i["tokens"], **on)
    pol = layers.policy_loss_forward(p.log_probs, i["old"], i["adv"], **on)
    d = layers.policy_loss_backward(p.log_probs, i["old"], i["adv"], pol.weights, **on)
    dl = layers.token_log_probs_backward(d, i["logits"], i["tokens"], p.lse, **on)
    got = [*o, *g, *h, *hg, *p, *pol, d, dl]
    torch.cuda.current_stream().wait_stream(s)
    got = [x.clone() for x in got if x is not None]
    o2 = layers.gated_scan_forward(i["gate"], i["x"], state=i["state"])
    g2 = layers.gated_scan_backward(o2.h, i["gate"], i["x"], o2.h, dstate=o2.state)
    h2 = layers.norm_rotate_heads_forward(q, q, i["w"], i["w"], cos=table[0], sin=table[1])
    hg2 = layers.norm_rotate_heads_backward(h2.q, h2.k, q, q, i["w"], i["w"], cos=table[0], sin=table[1])
    p2 = layers.token_log_probs_forward(i["logits"], i["tokens"])
    pol2 = layers.policy_loss_forward(p2.log_probs, i["old"], i["adv"])
    d2 = layers.policy_loss_backward(p2.log_probs, i["old"], i["adv"], pol2.weights)
    dl2 = layers.token_log_probs_backward(d2, i["logits"], i["tokens"], p2.lse)
    want = [x for x in [*o2, *g2, *h2, *hg2, *p2, *pol2, d2, dl2] if x is not None]
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_several_threads_at_once(layers):
    table = layers.rotation_table(200, 64)
    sets = [inputs(3, 200, v=700, seed=s) for s in range(4)]
    want = [[x.clone() for x in chain(layers, i, table)] for i in sets]
    torch.cuda.synchronize()
    wrong = []

    def work(k):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                got = chain(layers, sets[k], table)
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[k])):
                    wrong.append(k)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_inputs_are_left_as_they_were_and_results_are_apart(layers):
    table = layers.rotation_table(130, 64)
    i = inputs(3, 130)
    before = {k: v.clone() for k, v in i.items()}
    got = chain(layers, i, table)
    torch.cuda.synchronize()
    assert all(torch.equal(i[k], before[k]) for k in i)
    storages = [t.untyped_storage() for t in got]
    assert len({s.data_ptr() for s in storages}) == len(got)
    assert all(s.nbytes() == t.numel() * t.element_size() for t, s in zip(got, storages))


def test_second_derivatives_are_refused(layers):
    x = torch.randn(2, 6, 64, device="cuda", requires_grad=True)
    q = torch.randn(6, 2, 64, device="cuda", requires_grad=True)
    tokens = torch.zeros(2, 6, dtype=torch.int64, device="cuda")
    lp = torch.randn(2, 6, device="cuda", requires_grad=True)
    for y, leaf in ((layers.gated_scan(x, x).h, x), (layers.norm_rotate_heads(q).q, q),
                    (layers.token_log_probs(x, tokens), x),
                    (layers.policy_loss(lp, lp.detach(), lp.detach()).loss, lp)):
        (g,) = torch.autograd.grad((y * y).sum(), leaf, create_graph=True)
        with pytest.raises(RuntimeError):
            g.sum().backward()
