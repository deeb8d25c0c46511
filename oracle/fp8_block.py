"""FP8 (E4M3) KV blocks with one scale per (block, kv head), and the bookkeeping of one step
from request lengths, as their plain definitions (test infrastructure only).

The pages only say that serving engines store KV blocks in FP8 or INT4 (horeb.top "vLLM
PagedAttention：大模型推理的显存管理革命", section 生态现状); the readings here:

* a cache is codes [NB, Hkv, B, d] (uint8, E4M3 as in ``fp8``) and scales [NB, Hkv]; a code
  means decode(code) * scale;
* writing rows chooses e, the smallest integer with amax <= 448 * 2^e over the new rows of a
  (block, head), amax the largest finite magnitude, e held in [-100, 120].  A block whose
  row 0 is written takes 2^e; a block that already holds earlier rows takes the larger of
  2^e and its scale, and its earlier codes become E4M3(decode(code) * old / new);
* a new value becomes E4M3(x / scale), nearest, ties to even, infinities clamped, NaN kept;
* attention is ordinary attention over decode(code) * scale in float64.

A step's bookkeeping (``build_step``) gives each request ceil(context / B) blocks, the missing
ones from the head of the free list in request order, and each new token at position p the
slot table[p // B] * B + p % B.
"""
import numpy as np

from .attention import attend, validate_item
from .formats import decode_bits
from .fp8 import decode_e4m3, encode_e4m3

LOWEST, HIGHEST = -100, 120


def scale_exponent(amax):
    """The smallest integer e with amax <= 448 * 2^e, held in [LOWEST, HIGHEST]."""
    for e in range(LOWEST, HIGHEST):
        if amax <= np.ldexp(448.0, e):
            return e
    return HIGHEST


def _write_rows(codes, scales, b, h, a, rows):
    """Rows a .. of (block b, head h) := `rows` [m, d] (float64)."""
    finite = np.abs(rows[np.isfinite(rows)])
    new = np.ldexp(1.0, scale_exponent(finite.max() if finite.size else 0.0))
    if a > 0:
        old = float(scales[b, h])
        if new > old:
            codes[b, h, :a] = encode_e4m3(decode_e4m3(codes[b, h, :a]) * (old / new))
        else:
            new = old
    scales[b, h] = new
    codes[b, h, a:a + len(rows)] = encode_e4m3(rows / new)


def append(k8, v8, ks, vs, key_bits, value_bits, block_tables, context_lens, query_start, dtype):
    """Copies of the caches with each sequence's rows query_start[s] .. query_start[s+1]-1
    written at its positions context_lens[s] - q .. context_lens[s] - 1, and the set of error
    names met ("context", "block")."""
    out = [x.copy() for x in (k8, v8, ks, vs)]
    nb, hkv, B, _ = k8.shape
    T = block_tables.shape[1]
    errs = set()
    for s, c in enumerate(int(x) for x in context_lens):
        first, last = int(query_start[s]), int(query_start[s + 1])
        q = last - first
        if first < 0 or q < 0 or last > len(key_bits) or q > c or c > T * B:
            errs.add("context")
            continue
        p = c - q
        while p < c:
            stop = min(c, (p // B + 1) * B)
            b = int(block_tables[s, p // B])
            if 0 <= b < nb:
                at = slice(first + p - (c - q), first + stop - (c - q))
                for bits, codes, scales in ((key_bits, out[0], out[2]), (value_bits, out[1], out[3])):
                    x = decode_bits(bits[at], dtype)
                    for h in range(hkv):
                        _write_rows(codes, scales, b, h, p % B, x[:, h])
            else:
                errs.add("block")
            p = stop
    return (*out, errs)


def logical_rows(codes, scales, table_row, ctx):
    """Row t = decode(codes[table[t // B], :, t % B]) * scales[table[t // B]], float64."""
    B = codes.shape[2]
    out = np.empty((ctx,) + codes.shape[1:2] + codes.shape[3:])
    for t in range(ctx):
        b = int(table_row[t // B])
        out[t] = decode_e4m3(codes[b, :, t % B]) * scales[b].astype(np.float64)[:, None]
    return out


def paged_decode(q, k8, v8, ks, vs, block_tables, context_lens, scale):
    """q float64 [n, Hq, d] -> (out float64, error bits)."""
    outs, errs = np.zeros(q.shape), np.zeros(len(q), dtype=np.int64)
    for s in range(len(q)):
        ctx = int(context_lens[s])
        errs[s] = validate_item(block_tables[s], ctx, k8.shape[2], k8.shape[0])
        if not errs[s]:
            outs[s] = attend(q[s], logical_rows(k8, ks, block_tables[s], ctx),
                             logical_rows(v8, vs, block_tables[s], ctx), scale)
    return outs, errs


def paged_prefill(q, k8, v8, ks, vs, block_tables, context_lens, query_start, scale):
    """q float64 [rows, Hq, d]; the token at position p attends to 0 .. p.  -> out float64
    (zeros for a sequence that validate_item rejects or whose span exceeds its context)."""
    out = np.zeros(q.shape)
    for s in range(len(context_lens)):
        ctx, first, last = int(context_lens[s]), int(query_start[s]), int(query_start[s + 1])
        if last <= first or last - first > ctx or validate_item(block_tables[s], ctx, k8.shape[2], k8.shape[0]):
            continue
        k = logical_rows(k8, ks, block_tables[s], ctx)
        v = logical_rows(v8, vs, block_tables[s], ctx)
        for i in range(first, last):
            n = ctx - (last - 1 - i)
            out[i] = attend(q[i], k[:n], v[:n], scale)
    return out


def build_step(query_lens, context_lens, free_blocks, free_start, block_tables, block_size,
               num_blocks, num_slots):
    """-> (tables, slots, query_start, free_next, error names), everything copied."""
    B = block_size
    tables = np.array(block_tables)
    T = tables.shape[1]
    slots = np.full(num_slots, -1, dtype=np.int64)
    errs, plan, tokens, blocks = set(), [], 0, 0
    starts = [0]
    for q, c in zip((int(x) for x in query_lens), (int(x) for x in context_lens)):
        ok = 0 <= q <= c <= T * B
        if not ok:
            errs.add("context")
        have, need = (-(-(c - q) // B), -(-c // B) - -(-(c - q) // B)) if ok else (0, 0)
        plan.append((max(q, 0), c, ok, tokens, have, need, blocks))
        tokens += max(q, 0)
        blocks += need
        starts.append(min(tokens, 2 ** 31 - 1))
    if not 0 <= free_start <= len(free_blocks) or blocks > len(free_blocks) - free_start:
        errs.add("blocks")
    if tokens > num_slots:
        errs.add("slots")
    if errs & {"blocks", "slots"}:
        return tables, slots, np.array(starts, np.int32), free_start, errs
    for s, (q, c, ok, at, have, need, taken) in enumerate(plan):
        if not ok:
            continue
        row = [int(b) for b in tables[s, :have]]
        row += [int(b) for b in free_blocks[free_start + taken:free_start + taken + need]]
        for k in range(have, have + need):
            if 0 <= row[k] < num_blocks:
                tables[s, k] = row[k]
        for i in range(q):
            p = c - q + i
            if 0 <= row[p // B] < num_blocks:
                slots[at + i] = row[p // B] * B + p % B
            else:
                errs.add("block")
    return tables, slots, np.array(starts, np.int32), free_start + blocks, errs
