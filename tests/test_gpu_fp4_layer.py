"""One attention layer as a serving engine runs it: norm and rotation, the 4-bit
cache write, attention over the cache, for prompts in pieces and then token by
token, in eager calls and as a captured graph."""
import numpy as np
import pytest
import torch

import paged_kv_cache_group_b200 as fp8q
from gpu_util import dev, host
from oracle import fp4

pytestmark = pytest.mark.gpu

HEADS, GROUP, DIM, SIZE = 2, 4, 128, 16
Q_HEADS = HEADS * GROUP


class Layer:
    def __init__(self, batch, blocks, seed):
        g = torch.Generator().manual_seed(seed)
        self.kp, self.vp = fp8q.fp4_kv_pools(blocks, SIZE, HEADS, DIM)
        self.scales = torch.tensor([0.02, 0.03], device="cuda")
        self.freq = fp8q.rope_inv_freq(DIM, 1e6, 4.0, trained_length=4096)
        self.wq, self.wk = ((1 + 0.2 * torch.randn(DIM, generator=g)).to(torch.bfloat16).cuda()
                            for _ in range(2))

    def step(self, qkv, positions, slots, table, lens, start):
        x = qkv.unflatten(1, (-1, DIM))
        q, k, v = x[:, :Q_HEADS], x[:, Q_HEADS:Q_HEADS + HEADS], x[:, Q_HEADS + HEADS:]
        fp8q.qk_norm_rope(q, k, positions, self.freq, self.wq, self.wk, q_out=q, k_out=k)
        fp8q.fp4_kv_write(k, v, slots, self.kp, self.vp, scale_dev=self.scales)
        lse = torch.empty((qkv.shape[0], Q_HEADS), device="cuda")
        return fp8q.fp4_kv_attention(q, self.kp, self.vp, table, lens, q_start=start,
                                     scale_dev=self.scales, lse=lse)


def projections(seed, tokens):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((tokens, (Q_HEADS + 2 * HEADS) * DIM), generator=g).to(torch.bfloat16)


def reference(layer, history, table_row):
    """Attention of every token of one sequence, from the oracle: norm and
    rotation in 64 bits (the kernel's bf16 rows are within a rounding of them, so
    the cache itself is taken from the pool, checked against them)."""
    x = history.double().numpy().reshape(len(history), -1, DIM)
    pos = np.arange(len(history))
    f = layer.freq.cpu().numpy()
    q, _ = fp4.norm_rope(x[:, :Q_HEADS], pos, f, layer.wq.double().cpu().numpy(), 1e-6, False, 1.0)
    k, _ = fp4.norm_rope(x[:, Q_HEADS:Q_HEADS + HEADS], pos, f, layer.wk.double().cpu().numpy(), 1e-6,
                         False, 1.0)
    slots = table_row[pos // SIZE].astype(np.int64) * SIZE + pos % SIZE
    ks, vs = layer.scales.double().cpu().numpy()
    kc, vc = fp4.read(slots, host(layer.kp), "k") * ks, fp4.read(slots, host(layer.vp), "v") * vs
    # half a step of E2M1 is at most a sixth of the block's largest value, that
    # of its E4M3 scale a sixteenth: within 0.25 of it all together
    for cached, given in ((kc, k), (vc, x[:, Q_HEADS + HEADS:])):
        most = np.abs(given).reshape(*given.shape[:2], -1, 16).max(-1).repeat(16, -1)
        assert np.all(np.abs(cached - given) <= 0.25 * most + 1e-4)
    return fp4.attention(q, kc, vc, DIM ** -0.5, len(history))


def test_prompts_in_pieces_then_token_by_token():
    lengths = [70, 5, 33]
    steps = [[40, 5, 16], [30, 0, 17]] + [[1, 1, 1]] * 3
    layer = Layer(3, 30, 1)
    order = np.random.default_rng(2).permutation(30).astype(np.int32)
    table_host = np.stack([order[b * 6:b * 6 + 6] for b in range(3)])
    table = dev(table_host)
    data = [projections(10 + b, lengths[b] + 3) for b in range(3)]
    have = [0, 0, 0]
    outs = [[], [], []]
    for new in steps:
        rows, pos, slots, start = [], [], [], [0]
        for b, n in enumerate(new):
            p = np.arange(have[b], have[b] + n)
            rows.append(data[b][p])
            pos.append(p)
            slots.append(table_host[b, p // SIZE].astype(np.int64) * SIZE + p % SIZE)
            have[b] += n
            start.append(start[-1] + n)
        out, _ = layer.step(torch.cat(rows).cuda(), dev(np.concatenate(pos)), dev(np.concatenate(slots)),
                            table, dev(np.array(have, np.int32)), dev(np.array(start, np.int32)))
        for b in range(3):
            outs[b].append(out[start[b]:start[b + 1]].double().cpu().numpy())
    for b in range(3):
        want, _, mean, reach = reference(layer, data[b], table_host[b])
        got = np.concatenate(outs[b])
        # q is rounded to bf16 before the attention: 2^-8 of each product, at most
        # 2^-8 R in a score and twice that in a weight; then as the kernel's own
        # bound, whose smaller parts are below the 2^-9 added here
        bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -9 + 2.0 ** -7 * reach[..., None]) * mean
        assert np.all(np.abs(got - want) <= bound), float((np.abs(got - want) - bound).max())
    assert fp8q.fp8q_device_error(clear=True) == 0


def test_a_captured_decode_step_replayed():
    layers = [Layer(2, 20, 3), Layer(2, 20, 3)]
    table = dev(np.arange(20, dtype=np.int32).reshape(2, 10))
    fill = projections(30, 128).cuda()
    pos = torch.arange(64, device="cuda").repeat(2)
    slots = torch.cat([torch.arange(64), 160 + torch.arange(64)]).cuda()
    lens = torch.tensor([64, 64], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 64, 128], dtype=torch.int32, device="cuda")
    for layer in layers:
        layer.step(fill.clone(), pos, slots, table, lens, start)
    held = dict(qkv=torch.zeros((2, fill.shape[1]), dtype=torch.bfloat16, device="cuda"),
                positions=torch.zeros(2, dtype=torch.int64, device="cuda"),
                slots=torch.full((2,), -1, dtype=torch.int64, device="cuda"),
                lens=torch.ones(2, dtype=torch.int32, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layers[0].step(held["qkv"], held["positions"], held["slots"], table, held["lens"], None)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layers[0].step(held["qkv"], held["positions"], held["slots"], table, held["lens"], None)
    for i in range(40):                                       # over two block boundaries
        x = projections(40 + i, 2).cuda()
        p = torch.tensor([64 + i, 64 + i], device="cuda")
        s = p + torch.tensor([0, 160], device="cuda")
        n = (p + 1).to(torch.int32)
        for name, t in (("qkv", x), ("positions", p), ("slots", s), ("lens", n)):
            held[name].copy_(t)
        graph.replay()
        want = layers[1].step(x.clone(), p, s, table, n, None)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i
    assert torch.equal(layers[0].kp, layers[1].kp) and torch.equal(layers[0].vp, layers[1].vp)
    assert fp8q.fp8q_device_error(clear=True) == 0
