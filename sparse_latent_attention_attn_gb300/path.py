"""One step of the hot path, composed from the three C-ABI calls (marshalling only).

A decode step ("DeepSeek V4.1", attention/query-latent, Attention.forward with start_pos > 0):
  1. the new token's KV row is rounded through fp8 in place and stored to ring slot
     start_pos % window ("Module attn", act_quant_inplace and the ring-cache paragraph);
  2. the window columns of the index rows are written: the whole ring, oldest first
     ("DeepSeek V4.1", attention/attend, get_window_topk_idxs);
  3. sparse_attn over kv = [ring | compressed rows] with idx = [window cols | compressed cols].

A prefill step at start_pos 0 rounds the whole chunk in place (it is also the window part of kv
for this step), keeps its last `window` rows in the ring, writes one causal window row per query
and runs sparse_attn over kv = [chunk | compressed rows].

A decode step over the paged 4-bit row store has every sequence at a position of its own: the new
row is normalised, rotated and stored as codes in its ring slot, the queries are normalised and rotated,
and sparse_attn runs over the listed rows of the store with its output rotated back.

A step over the paged 8-bit row store takes a chunk of one or many new tokens of every sequence, a prompt's next piece as
well as a decode step, in a layer where a query sees its window and every complete compressed row (while there are
no more of those than the Indexer would keep, or in a layer without them): no index rows are made.

The caller lays kv out as [window rows | compressed rows] per sequence and idx as
[window cols | compressed cols], so no concatenation copy is made.
"""
from __future__ import annotations

import torch

from . import dsattn


def decode_step(q: torch.Tensor, kv: torch.Tensor, new_kv: torch.Tensor, sink: torch.Tensor, idx: torch.Tensor,
                start_pos: int, window: int, scale: float, o: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q [b][1][h][d]; kv [b][window + C][d] (ring first); new_kv [b][1][d] raw row of this token
    (rounded in place); idx [b][1][window + K] with the compressed columns already filled."""
    b = q.shape[0]
    dsattn.kv_quant_ring_write(new_kv, kv[:, :window], start_pos, window, stream=stream)
    dsattn.window_topk_idxs(idx, b, 1, start_pos, window, stream=stream)
    return dsattn.sparse_attn(q, kv, sink, idx, scale, o=o, workspace=workspace, stream=stream)


def prefill_step(q: torch.Tensor, kv: torch.Tensor, ring: torch.Tensor, sink: torch.Tensor, idx: torch.Tensor,
                 window: int, scale: float, o: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                 stream=None, pairs: bool = False) -> torch.Tensor:
    """q [b][s][h][d]; kv [b][s + C][d] (the raw chunk first, rounded in place); ring [b][window][d];
    idx [b][s][min(s, window) + K] with the compressed columns already filled.  pairs: neighbouring
    queries share one gather (ds_sparse_attn_prefill; its own workspace size)."""
    b, s = q.shape[0], q.shape[1]
    dsattn.kv_quant_ring_write(kv[:, :s], ring, 0, window, stream=stream)
    dsattn.window_topk_idxs(idx, b, s, 0, window, stream=stream)
    if pairs:
        return dsattn.sparse_attn_prefill(q, kv, sink, idx, scale, o=o, workspace=workspace, stream=stream)
    return dsattn.sparse_attn(q, kv, sink, idx, scale, o=o, workspace=workspace, stream=stream)


def decode_step_fp4_paged(q: torch.Tensor, new_kv: torch.Tensor, codes: torch.Tensor, exps: torch.Tensor,
                          block_table: torch.Tensor, first: torch.Tensor, sink: torch.Tensor, idx: torch.Tensor,
                          window: int, scale: float, rd: int, table: torch.Tensor, eps: float,
                          kv_weight: torch.Tensor | None = None, lens: torch.Tensor | None = None,
                          o: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """q [b][s][h][d] and new_kv [b][s][d] as their projections leave them (neither is modified); the token
    (bi, t) is at position first[bi] + t; codes, exps, block_table: the paged store, whose logical rows
    are the ring's `window` slots, then the compressed rows; idx [b][s][topk] lists logical rows, complete.
    Tokens at or behind lens[bi] are padding: nothing of theirs is stored, and o is left as it was (zeros in a
    new one).  s > 1 stores all s rows before any query reads them, so the ring has to hold what every query of the step
    lists: `window` = (the rows a query attends over) + s - 1 slots.  Fewer slots than tokens, which would not
    keep the step's own rows, are refused (with lens, which must not exceed them either, they cannot be told);
    window = 0 is a cache without a ring (row = position)."""
    if lens is None and 0 < window < q.shape[1]:
        raise ValueError(f"a ring of {window} slots does not hold the step's {q.shape[1]} tokens")
    dsattn.kv_append_fp4_paged(new_kv, codes, exps, block_table, first, rd=rd, table=table, eps=eps, weight=kv_weight,
                               lens=lens, window=window, stream=stream)
    qn = None
    if lens is not None:                   # the padding of q is not read: no zeros for it
        with dsattn._on(stream):
            qn = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    qn = dsattn.norm_rotary(q, eps, rd, table, first, lens=lens, y=qn, stream=stream)
    return dsattn.sparse_attn_fp4_paged(qn, codes, exps, block_table, sink, idx, scale, rd=rd, table=table,
                                        first=first, o=o, workspace=workspace, stream=stream, lens=lens)


def chunk_step_fp8_paged(q: torch.Tensor, new_kv: torch.Tensor, codes: torch.Tensor, exps: torch.Tensor,
                         block_table: torch.Tensor, first: torch.Tensor, sink: torch.Tensor, window: int, ring: int,
                         scale: float, rd: int, table: torch.Tensor, eps: float, kv_weight: torch.Tensor | None = None,
                         lens: torch.Tensor | None = None, ratio: int = 0, base: int = 0,
                         o: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q [b][s][h][d] and new_kv [b][s][d] as their projections leave them (neither is modified); the token (bi, t) is at
    position first[bi] + t.  Its row is normalised, rotated and stored as e4m3 codes (in slot position % ring of the
    ring, or at its position for ring = 0), and its queries see the last `window` positions (0: all) and, with
    ratio > 0, the compressed rows of every complete group of `ratio` positions, which are in the store from logical row
    `base` on (kv_append_fp8_paged with pos_step = ratio and that base).  Tokens at or behind lens[bi] are
    padding: nothing of theirs is stored, and o is left as it was (zeros in a new one).  The ring must hold
    window + s - 1 rows (with lens: window + the largest of them - 1) and lie in the block table, before the compressed rows;
    one that does not is refused before anything is stored in it."""
    s = q.shape[1]
    if ring > 0 and (window <= 0 or ring < window + (max(s, 1) - 1 if lens is None else 0)):
        raise ValueError(f"a ring of {ring} slots does not hold a window of {window} and the step's {s} tokens")
    if ring > 0 and codes.dim() == 3 and (ring > codes.shape[1] * block_table.shape[-1] or (ratio > 0 and base < ring)):
        raise ValueError(f"a ring of {ring} slots does not fit into {block_table.shape[-1]} pages of {codes.shape[1]} rows, "
                         f"before the compressed rows from {base} on")
    dsattn.kv_append_fp8_paged(new_kv, codes, exps, block_table, first, rd=rd, table=table, eps=eps, weight=kv_weight,
                               lens=lens, window=ring, stream=stream)
    qn = None
    if lens is not None:                   # the padding of q is not read: no zeros for it
        with dsattn._on(stream):
            qn = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    qn = dsattn.norm_rotary(q, eps, rd, table, first, lens=lens, y=qn, stream=stream)
    return dsattn.chunk_attn_fp8_paged(qn, codes, exps, block_table, first, sink, scale, window, ring=ring, ratio=ratio,
                                       base=base, lens=lens, rd=rd, table=table, o=o, workspace=workspace, stream=stream)
