"""The calls of a serving step one behind the other, as an engine makes them: norms, rotation and store
of the new tokens (kv_append), their attention in chunks (paged_chunk_attn), then single tokens
(paged_decode_attn_sinks), over blocks that a BlockManager hands out, with a window and sinks; in
a captured graph; on two host threads; over a pool of more than 4 GiB."""
import threading

import pytest
import torch

import heads_plain as P
import paged_kv_attention_22_gb300 as pkv
from attn_plain import SCALE, attend, seen
from paged_kv_attention_22_gb300 import build as pkv_build

DEV = "cuda"
Hq, H, BS = 8, 4, 32
WINDOW, SINKS = 50, 5


@pytest.fixture(scope="module")
def L():
    pkv_build.build()
    return pkv.lib()


class Layer:
    """One layer's weights, cache and rotation, and its projections of every token of `lengths`."""

    def __init__(self, lengths, num_blocks, seed, window=WINDOW, sinks=SINKS):
        g = torch.Generator().manual_seed(seed)
        self.tokens = [torch.randn(n, (Hq + 2 * H) * 128, generator=g).to(torch.bfloat16).to(DEV) for n in lengths]
        self.wq, self.wk = ((1 + 0.3 * torch.randn(128, generator=g)).to(torch.bfloat16).to(DEV) for _ in range(2))
        self.kc, self.vc = (torch.full((num_blocks, BS, H, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
                            for _ in range(2))
        self.rope = pkv.rope(96, base=1e6, scaling="ntk", factor=2.0)
        self.window, self.sinks = window, sinks

    def heads(self, rows):
        """q, k, v of rows of projections, as views of them."""
        q, k, v = rows.split([Hq * 128, H * 128, H * 128], 1)
        return q.unflatten(1, (Hq, 128)), k.unflatten(1, (H, 128)), v.unflatten(1, (H, 128))

    def append(self, rows, positions, slots):
        q, k, v = self.heads(rows)
        return pkv.kv_append(q, k, v, self.rope, positions, self.kc, self.vc, slots, self.wq, self.wk, eps=1e-5)

    def check_rows(self, s, q, first, slots):
        """q and the cache's rows of sequence s's tokens from `first` on against the plain form."""
        n = q.shape[0]
        qs, ks, vs = self.heads(self.tokens[s][first:first + n])
        pos = torch.arange(first, first + n, dtype=torch.int32, device=DEV)
        f, m = P.frequencies(96, 1e6, "ntk", factor=2.0)
        flat = lambda c: c.flatten(0, 1)[slots.long()]
        for got, x, w in ((q, qs, self.wq), (flat(self.kc), ks, self.wk)):
            want, tol = P.turned(x, w, pos, 96, f, m, False, eps=1e-5)
            assert bool(((got.double().cpu() - want).abs() <= tol).all())
        assert torch.equal(flat(self.vc).view(torch.int16), vs.contiguous().view(torch.int16))

    def check_attention(self, q, out, lse, slots, last, rounded):
        """out and lse of q at positions `last` over the sequence's cached rows, at `slots`."""
        k, v = (c.flatten(0, 1)[slots.long()] for c in (self.kc, self.vc))
        mask = seen(last, k.shape[0], self.window, self.sinks)
        want, wl, tol, ltol = attend(q, k, v, mask, SCALE, rounded)
        assert bool(((out.double().cpu() - want).abs() <= tol).all())
        assert bool(((lse.double().cpu() - wl).abs() <= ltol).all())


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _slots(m, s, first, count):
    return torch.as_tensor(m.slots(s, first, count) if count else []).to(torch.int32).to(DEV)


@pytest.mark.gpu
def test_prompts_in_pieces_then_single_tokens(L):
    prompts, steps = [200, 3, 130], 6
    layer = Layer([n + steps for n in prompts], 40, seed=1)
    m = pkv.BlockManager(40, BS)
    ids = list(range(3))
    for s, n in enumerate(prompts):
        m.add_sequence(s, [1000 * s + t for t in range(n)])
    width = 8
    ws, dws = pkv.new_chunk_workspace(3, Hq, H), pkv.new_decode_workspace(3, Hq, H, 128, 256)
    done = [0, 0, 0]
    for piece in (70, 70, 70):  # each sequence's next 70 tokens, as far as it has them
        new = [min(piece, n - d) for n, d in zip(prompts, done)]
        rows = torch.cat([layer.tokens[s][done[s]:done[s] + new[s]] for s in ids])
        pos = torch.cat([torch.arange(done[s], done[s] + new[s]) for s in ids]).to(torch.int32).to(DEV)
        q = layer.append(rows, pos, torch.cat([_slots(m, s, done[s], new[s]) for s in ids]))
        cu = _ints([0] + new).cumsum(0).to(torch.int32)
        lens = [d + n for d, n in zip(done, new)]
        bt = torch.as_tensor(m.block_tables(ids, width)).to(torch.int32).to(DEV)
        out, lse = pkv.paged_chunk_attn(q, layer.kc, layer.vc, cu, _ints(lens), bt, max(new), max(lens), SCALE,
                                        sliding_window=WINDOW, num_sinks=SINKS, workspace=ws)
        at = 0
        for s in ids:
            part = slice(at, at + new[s])
            if new[s]:
                layer.check_rows(s, q[part], done[s], _slots(m, s, done[s], new[s]))
                layer.check_attention(q[part], out[part], lse[part], _slots(m, s, 0, lens[s]),
                                      list(range(done[s], lens[s])), True)
            at += new[s]
        done = lens
    for step in range(steps):
        for s in ids:
            m.append_token(s, 5000 + step)
        rows = torch.stack([layer.tokens[s][done[s]] for s in ids])
        slots = torch.cat([_slots(m, s, done[s], 1) for s in ids])
        q = layer.append(rows, _ints(done), slots)
        done = [d + 1 for d in done]
        bt = torch.as_tensor(m.block_tables(ids, width)).to(torch.int32).to(DEV)
        out, lse = pkv.paged_decode_attn_sinks(q, layer.kc, layer.vc, bt, _ints(done), max(done), SCALE, WINDOW, SINKS,
                                               workspace=dws)
        again = pkv.paged_chunk_attn(q, layer.kc, layer.vc, _ints([0, 1, 2, 3]), _ints(done), bt, 1, max(done), SCALE,
                                     sliding_window=WINDOW, num_sinks=SINKS, workspace=ws)
        for s in ids:
            part = slice(s, s + 1)
            layer.check_rows(s, q[part], done[s] - 1, slots[part])
            whole = _slots(m, s, 0, done[s])
            layer.check_attention(q[part], out[part], lse[part], whole, [done[s] - 1], False)
            layer.check_attention(q[part], again[0][part], again[1][part], whole, [done[s] - 1], True)
    assert pkv.check_device_errors() == 0


@pytest.mark.gpu
def test_a_captured_step_replayed_as_sequences_grow(L):
    # two layers in one graph share the decode workspace; a second graph, of the chunk call, its own
    start, steps = [40, 7], 40
    layers = [Layer([n + steps for n in start], 12, seed=2 + i) for i in range(2)]
    bt = _ints([[3, 7, 1, 0], [5, 2, 9, 4]])
    slot = lambda s, t: int(bt[s, t // BS]) * BS + t % BS
    all_slots = [_ints([slot(s, t) for t in range(n + steps)]) for s, n in enumerate(start)]
    for layer in layers:
        for s, n in enumerate(start):
            layer.append(layer.tokens[s][:n], _ints(list(range(n))), all_slots[s][:n])
    rows = [torch.zeros(2, (Hq + 2 * H) * 128, dtype=torch.bfloat16, device=DEV) for _ in layers]
    pos, slots, lens = _ints([0, 0]), _ints([0, 0]), _ints([1, 1])
    cu = _ints([0, 1, 2])
    ws, cws = pkv.new_decode_workspace(2, Hq, H, 128, 128), pkv.new_chunk_workspace(2, Hq, H)
    graphs, results = [torch.cuda.CUDAGraph() for _ in range(2)], [[], []]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graphs[0], stream=side):
        for layer, x in zip(layers, rows):
            q = layer.append(x, pos, slots)
            results[0].append((q, *pkv.paged_decode_attn_sinks(q, layer.kc, layer.vc, bt, lens, 128, SCALE, WINDOW,
                                                               SINKS, workspace=ws)))
    with torch.cuda.graph(graphs[1], stream=side):
        for layer, (q, _, _) in zip(layers, results[0]):
            results[1].append((q, *pkv.paged_chunk_attn(q, layer.kc, layer.vc, cu, lens, bt, 1, 128, SCALE,
                                                        sliding_window=WINDOW, num_sinks=SINKS, workspace=cws)))
    for step in range(steps):
        at = [n + step for n in start]
        pos.copy_(_ints(at))
        lens.copy_(_ints([t + 1 for t in at]))
        slots.copy_(_ints([slot(s, t) for s, t in enumerate(at)]))
        for layer, x in zip(layers, rows):
            x.copy_(torch.stack([layer.tokens[s][t] for s, t in enumerate(at)]))
        graphs[0].replay()
        graphs[1].replay()
        if step % 13:
            continue
        torch.cuda.synchronize()
        for layer, decoded, chunked in zip(layers, *results):
            for s, t in enumerate(at):
                for (q, out, lse), rounded in ((decoded, False), (chunked, True)):
                    layer.check_attention(q[s:s + 1], out[s:s + 1], lse[s:s + 1], all_slots[s][:t + 1], [t], rounded)
    assert pkv.check_device_errors() == 0


@pytest.mark.gpu
def test_two_host_threads(L):
    def work(seed, stream, results):
        with torch.cuda.stream(stream):
            layer = Layer([700], 30, seed=seed)
            slots, bt = torch.arange(700, dtype=torch.int32, device=DEV), _ints([list(range(22))])
            dws, cws = pkv.new_decode_workspace(1, Hq, H, 128, 700), pkv.new_chunk_workspace(1, Hq, H)
            for _ in range(20):
                q = layer.append(layer.tokens[0], slots, slots)
                a = pkv.paged_chunk_attn(q[:690], layer.kc, layer.vc, _ints([0, 690]), _ints([690]), bt, 690, 700, SCALE,
                                         sliding_window=WINDOW, num_sinks=SINKS, workspace=cws)
                b = pkv.paged_decode_attn_sinks(q[699:], layer.kc, layer.vc, bt, _ints([700]), 700, SCALE, WINDOW, SINKS,
                                                workspace=dws)
                results.append((q, *a, *b))
            stream.synchronize()

    alone, together = [[], []], [[], []]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        work(20 + i, streams[i], alone[i])
    threads = [threading.Thread(target=work, args=(20 + i, streams[i], together[i])) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for one, both in zip(alone, together):
        assert len(both) == 20
        for x, y in zip(one, both):
            assert all(torch.equal(a, b) for a, b in zip(x, y))
    assert pkv.check_device_errors() == 0


@pytest.mark.gpu
def test_a_pool_of_more_than_4_gib(L):
    blocks = (1 << 32) // (BS * H * 256) + 20
    layer = Layer([], 1, seed=6)
    layer.kc, layer.vc = (torch.empty(blocks, BS, H, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    assert layer.kc.numel() * 2 > 1 << 32
    g = torch.Generator().manual_seed(7)
    layer.tokens = [torch.randn(300, (Hq + 2 * H) * 128, generator=g).to(torch.bfloat16).to(DEV)]
    bt = _ints([[blocks - 1 - j if j % 2 else j for j in range(10)]])  # at both ends
    slots = (bt[0].long()[:, None] * BS + torch.arange(BS, device=DEV)).flatten()[:300].to(torch.int32)
    q = layer.append(layer.tokens[0], torch.arange(300, dtype=torch.int32, device=DEV), slots)
    layer.check_rows(0, q, 0, slots)
    out, lse = pkv.paged_chunk_attn(q[250:], layer.kc, layer.vc, _ints([0, 50]), _ints([300]), bt, 50, 300, SCALE,
                                    sliding_window=WINDOW, num_sinks=SINKS)
    layer.check_attention(q[250:], out, lse, slots, list(range(250, 300)), True)
    out, lse = pkv.paged_decode_attn_sinks(q[299:], layer.kc, layer.vc, bt, _ints([300]), 300, SCALE, WINDOW, SINKS)
    layer.check_attention(q[299:], out, lse, slots, [299], False)
    layer.window = 0
    out, lse = pkv.paged_chunk_attn(q, layer.kc, layer.vc, _ints([0, 300]), _ints([300]), bt, 300, 300, SCALE)
    layer.check_attention(q, out, lse, slots, list(range(300)), True)
    assert pkv.check_device_errors() == 0
