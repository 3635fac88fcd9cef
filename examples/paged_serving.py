"""One attention layer of a served model over a paged cache, with its pages
moved out to host memory and back between two turns of a conversation.

    python examples/paged_serving.py [--format fp8|int8|bf16] [--prompt N] [--chunk N] [--new N]

Two sequences are prefilled chunk by chunk: rotary positions (kvcache.rope),
the new keys and values into pages (kvcache.write), attention over the pages
(kvcache.AttentionPlan).  The first sequence's pages then go to mapped host
memory in one kvcopy_batch, as a connector parks an idle conversation, come
back into other pages, and both sequences decode single tokens.  The same is
done without the trip to the host, and the outputs have to be equal bit for
bit: neither the place of a page nor its way there changes a result.

Queries, keys and values are random (there are no weights); sizes are those of
a layer with 32 query heads and 8 key/value heads of 128.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from block_copy_amd import kvcache as C  # noqa: E402
from block_copy_amd import kvcopy as K  # noqa: E402

HEADS, KV_HEADS, DIM, PAGE = 32, 8, 128, 16
DTYPES = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}


class Layer:
    """A paged cache and the page lists of the sequences in it."""

    def __init__(self, pages, fmt, device):
        dt = DTYPES[fmt]
        shape = (pages, KV_HEADS, PAGE, DIM)
        self.k, self.v = (torch.zeros(shape, dtype=torch.uint8 if dt.itemsize == 1 else dt, device=device).view(dt)
                          for _ in range(2))
        scales = [torch.zeros(shape[:3], device=device) for _ in range(2)] if dt.itemsize == 1 else [None, None]
        self.cache = C.PagedCache(self.k, self.v, *scales)
        self.parts = [self.k, self.v] + [s for s in scales if s is not None]
        self.device = device
        self.free = list(range(pages))
        self.pages, self.lengths = {}, {}
        # contexts eight times as long as the frequencies' own: slow waves slowed
        self.freqs = C.rope_frequencies(DIM, 500000.0, "parts", factor=8.0, original=8192, device=device)

    def step(self, rows):
        """rows: {sequence: (q, k, v)} of new tokens.  Returns their outputs."""
        for s, (q, _, _) in rows.items():
            have = self.lengths.get(s, 0) + q.shape[0]
            mine = self.pages.setdefault(s, [])
            while len(mine) * PAGE < have:
                mine.append(self.free.pop())
        seqs = list(rows)
        lens = [rows[s][0].shape[0] for s in seqs]
        old = [self.lengths.get(s, 0) for s in seqs]
        ctx = [o + n for o, n in zip(old, lens)]
        positions = torch.cat([torch.arange(o, c) for o, c in zip(old, ctx)])
        slots = torch.cat([torch.tensor(self.pages[s])[torch.arange(o, c) // PAGE] * PAGE + torch.arange(o, c) % PAGE
                           for s, o, c in zip(seqs, old, ctx)])
        table = torch.zeros(len(seqs), max(len(self.pages[s]) for s in seqs), dtype=torch.int32)
        for i, s in enumerate(seqs):
            table[i, :len(self.pages[s])] = torch.tensor(self.pages[s], dtype=torch.int32)
        starts = torch.tensor([0] + lens).cumsum(0)
        q, k, v = (torch.cat([rows[s][j] for s in seqs]) for j in range(3))
        d = self.device

        q, k = C.rope(positions.to(torch.int32).to(d), self.freqs, q, k)
        C.write(self.cache, k, v, slots.to(d))
        plan = C.AttentionPlan(self.cache, q_heads=HEADS, num_seqs=len(seqs), total_q=sum(lens), max_q_len=max(lens),
                               max_context=max(ctx), dtype=q.dtype)
        out = plan(q, table.to(d), starts.to(torch.int32).to(d), torch.tensor(ctx, dtype=torch.int32, device=d))
        for s, c in zip(seqs, ctx):
            self.lengths[s] = c
        return dict(zip(seqs, out.split(lens)))

    def _blocks(self, pages, base):
        """(device address, host address, size) of every part of the pages."""
        dev, host, size = [], [], []
        for part in self.parts:
            block = part[0].numel() * part.element_size()
            for p in pages:
                dev.append(part.data_ptr() + p * block)
                host.append(base + sum(size))
                size.append(block)
        return dev, host, size

    def park(self, s):
        """The sequence's pages to host memory; frees and overwrites them."""
        pages = self.pages[s]
        total = sum(self._blocks(pages, 0)[2])
        buffer = K.HostBuffer(total)
        dev, host, size = self._blocks(pages, buffer.ptr)
        stream = torch.cuda.current_stream(self.device)
        K.kvcopy_batch(dev, host, size, K.D2H, K.WGS_AUTO, stream.cuda_stream)
        stream.synchronize()
        for part in self.parts:
            (part.view(torch.uint8) if part.element_size() == 1 else part)[pages] = 0
        self.free = pages + self.free      # handed out last: the sequence comes back elsewhere
        del self.pages[s]
        return buffer, len(pages)

    def resume(self, s, parked):
        buffer, n = parked
        self.pages[s] = [self.free.pop() for _ in range(n)]
        dev, host, size = self._blocks(self.pages[s], buffer.ptr)
        stream = torch.cuda.current_stream(self.device)
        K.kvcopy_batch(host, dev, size, K.H2D, K.WGS_AUTO, stream.cuda_stream)
        stream.synchronize()
        buffer.free()


def serve(fmt, prompt, chunk, new, move, device="cuda:0"):
    """The outputs of every step; `move`: sequence 0 goes to the host and back
    between the prompt and the new tokens."""
    device = torch.device(device)
    g = torch.Generator(device=device)
    g.manual_seed(7)
    lengths = {0: prompt, 1: max(1, prompt // 3)}
    layer = Layer(3 * (-(-(prompt + new) // PAGE)) + 8, fmt, device)

    def fresh(n):
        return [torch.randn(n, h, DIM, device=device, generator=g).to(torch.bfloat16) for h in (HEADS, KV_HEADS, KV_HEADS)]

    outs = []
    left = dict(lengths)
    while any(left.values()):
        rows = {s: fresh(min(chunk, n)) for s, n in left.items() if n}
        left = {s: n - (rows[s][0].shape[0] if s in rows else 0) for s, n in left.items()}
        outs += list(layer.step(rows).values())
    before = list(layer.pages[0])
    if move:
        layer.resume(0, layer.park(0))
        assert set(before) != set(layer.pages[0])
    for _ in range(new):
        outs += list(layer.step({s: fresh(1) for s in lengths}).values())
    torch.cuda.synchronize(device)
    return outs


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--format", choices=sorted(DTYPES), default="fp8")
    ap.add_argument("--prompt", type=int, default=3000)
    ap.add_argument("--chunk", type=int, default=512)
    ap.add_argument("--new", type=int, default=16)
    a = ap.parse_args(argv)
    stay = serve(a.format, a.prompt, a.chunk, a.new, move=False)
    moved = serve(a.format, a.prompt, a.chunk, a.new, move=True)
    same = all(torch.equal(x, y) for x, y in zip(stay, moved))
    finite = all(bool(x.isfinite().all()) for x in stay)
    print(f"{a.format}: {len(stay)} outputs, {sum(x.shape[0] for x in stay)} tokens; "
          f"with the first sequence moved to the host and back: {'the same bits' if same else 'DIFFERENT'}")
    return 0 if same and finite and len(stay) == len(moved) else 1


if __name__ == "__main__":
    sys.exit(main())
