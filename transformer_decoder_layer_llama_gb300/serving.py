"""Continuous batching over a stack of decoder layers on one GPU.

Host-side logic from the pages, driving the C-ABI layer calls:

* paged KV-cache management (page "ATB KV-cache paging, quantisation,
  speculative decoding and communication overlap", section "KV Cache memory
  wall"): fixed-size blocks handed out on demand from a free list, a
  block_table per request mapping its logical blocks to physical ones, blocks
  of a finished request returned to the free list at once and reused in any
  order;
* the continuous-batching scheduler (page "ATB: whole decoder-layer fusion",
  section "graph execution engine"): a running set of requests, each step
  allocating what every request needs (a KV slot) and recycling a finished
  request's resources immediately to admit a new one.

One block table serves every layer: layer l keeps its own K/V pool, indexed by
the same physical block ids.  Each step first prefills the newly admitted
requests (all layers, one batched prefill call per layer), then runs one decode
step for every slot through all layers (one decode call per layer; this part
can be captured once as a CUDA graph and replayed with the tables updated in
place).  Every computation runs in the library's kernels; this module only
moves indices.

Requests can share blocks: a fork shares its parent's full blocks (each block
counts its holders, and returns to the free list when the last one lets go) and
copies the block that is still filling, in the pools of every layer at once.
After many admissions and retirements the blocks in use can be packed to the
front of the pools.
"""
from __future__ import annotations

import dataclasses

import numpy as np
import torch

from . import synth


class BlockAllocator:
    """LIFO free list of physical KV blocks (seeded initial order), with the number of holders of each
    block in use."""

    def __init__(self, num_blocks: int, seed: int):
        g = torch.Generator()
        g.manual_seed(int(seed))
        self.num_blocks = int(num_blocks)
        self._free = torch.randperm(self.num_blocks, generator=g).tolist()
        self._used = {}

    def free_count(self) -> int:
        return len(self._free)

    def holders(self, block: int) -> int:
        return self._used.get(block, 0)

    def in_use(self) -> list:
        return list(self._used)

    def alloc(self, n: int) -> list:
        if n > len(self._free):
            raise MemoryError(f"KV pool exhausted: need {n} blocks, {len(self._free)} free")
        out = [self._free.pop() for _ in range(n)]
        self._used.update((b, 1) for b in out)
        return out

    def share(self, blocks) -> None:
        """One more holder for each of the blocks."""
        blocks = list(blocks)
        for b in blocks:
            if b not in self._used:
                raise ValueError(f"block {b} is not in use")
        for b in blocks:
            self._used[b] += 1

    def free(self, blocks) -> None:
        """One holder less; a block without any returns to the free list."""
        for b in blocks:
            if b not in self._used:
                raise ValueError(f"block {b} freed twice or never allocated")
            self._used[b] -= 1
            if self._used[b] == 0:
                del self._used[b]
                self._free.append(b)

    def apply_map(self, block_map) -> None:
        """Renames the blocks in use as compact_blocks' block_map says (old id -> new id, -1: not in use)."""
        moved = {int(block_map[b]): n for b, n in self._used.items()}
        if len(moved) != len(self._used) or any(not 0 <= b < self.num_blocks for b in moved):
            raise ValueError("the map does not name every block in use")
        self._used = moved
        self._free = [b for b in range(self.num_blocks - 1, -1, -1) if b not in moved]


@dataclasses.dataclass
class Request:
    rid: int
    ctx: int              # tokens in the cache
    budget: int           # decode tokens still to produce
    blocks: list


class Scheduler:
    """Slots, budgets and the block table (host side, numpy)."""

    def __init__(self, n_slots: int, block_size: int, max_blocks: int, allocator: BlockAllocator,
                 seed: int, budget_max: int = 256, prompt_len: int = 256):
        self.n_slots, self.bs, self.max_blocks = n_slots, block_size, max_blocks
        self.alloc = allocator
        self.prompt_len, self.budget_max = prompt_len, budget_max
        self.rng = np.random.default_rng(seed)
        self.table = np.full((n_slots, max_blocks), -1, np.int32)
        self.slots: list = [None] * n_slots
        self.next_rid = 0

    def _new_budget(self) -> int:
        return int(self.rng.integers(1, self.budget_max + 1))

    def _set_blocks(self, slot: int, blocks: list) -> None:
        if len(blocks) > self.max_blocks:
            raise ValueError("request outgrew the block table width")
        self.table[slot, :] = -1
        self.table[slot, :len(blocks)] = blocks

    def start_resident(self, slot: int, ctx: int) -> Request:
        """A request whose first `ctx` tokens are already cached (pre-filled pool)."""
        blocks = self.alloc.alloc(-(-ctx // self.bs))
        r = Request(self.next_rid, ctx, self._new_budget(), blocks)
        self.next_rid += 1
        self.slots[slot] = r
        self._set_blocks(slot, blocks)
        return r

    def retire_and_admit(self) -> list:
        """Frees every finished request's blocks and admits a new request in its slot.
        Returns the slots that need a prefill of `prompt_len` tokens this step."""
        admitted = []
        for s, r in enumerate(self.slots):
            if r is not None and r.budget > 0:
                continue
            if r is not None:
                self.alloc.free(r.blocks)
            blocks = self.alloc.alloc(-(-self.prompt_len // self.bs))
            nr = Request(self.next_rid, self.prompt_len, self._new_budget(), blocks)
            self.next_rid += 1
            self.slots[s] = nr
            self._set_blocks(s, blocks)
            admitted.append(s)
        return admitted

    def retire(self, slot: int) -> None:
        """Ends the request in a slot now: its blocks are let go, the slot is empty until the next fork into it,
        start_resident or retire_and_admit."""
        r = self.slots[slot]
        if r is None:
            raise ValueError(f"slot {slot} is empty")
        self.alloc.free(r.blocks)
        self.slots[slot] = None
        self.table[slot, :] = -1

    def fork(self, src: int, dst: int) -> list:
        """A copy of the request in slot `src` for the empty slot `dst`: full blocks are shared, the one that is
        still filling is copied.  Returns the (from, to) block pairs to copy in every pool before either
        request goes on."""
        r = self.slots[src]
        if r is None or self.slots[dst] is not None:
            raise ValueError(f"a fork goes from a request to an empty slot, not from slot {src} to {dst}")
        full = r.ctx // self.bs
        last = self.alloc.alloc(1) if r.ctx % self.bs else []
        self.alloc.share(r.blocks[:full])
        nr = Request(self.next_rid, r.ctx, r.budget, r.blocks[:full] + last)
        self.next_rid += 1
        self.slots[dst] = nr
        self._set_blocks(dst, nr.blocks)
        return [(r.blocks[full], last[0])] if last else []

    def held_outside(self) -> list:
        """Blocks in use that somebody besides the requests in the slots holds (a prefix kept with share, blocks
        from alloc): a renaming reaches the requests' ids only."""
        mine = {}
        for r in self.slots:
            for b in r.blocks if r is not None else ():
                mine[b] = mine.get(b, 0) + 1
        return sorted(b for b in self.alloc.in_use() if self.alloc.holders(b) != mine.get(b, 0))

    def apply_map(self, block_map) -> None:
        """Renames every block as compact_blocks' block_map says."""
        self.alloc.apply_map(block_map)
        for s, r in enumerate(self.slots):
            if r is not None:
                r.blocks = [int(block_map[b]) for b in r.blocks]
                self._set_blocks(s, r.blocks)

    def grow_for_decode(self) -> np.ndarray:
        """Every slot appends one token: a block is added when the new position starts one.
        Returns context_lens (int32) including the appended token.  A decode step has a request in every slot
        (fork, start_resident or retire_and_admit fill one that retire left empty): with an empty one ValueError, with
        too few free blocks MemoryError, and no request is changed."""
        empty = [s for s, r in enumerate(self.slots) if r is None]
        if empty:
            raise ValueError(f"slots {empty} are empty")
        new = [s for s, r in enumerate(self.slots) if r.ctx % self.bs == 0 and r.ctx // self.bs >= len(r.blocks)]
        if any(len(self.slots[s].blocks) >= self.max_blocks for s in new):
            raise ValueError("request outgrew the block table width")
        for s, b in zip(new, self.alloc.alloc(len(new))):
            r = self.slots[s]
            r.blocks.append(b)
            self._set_blocks(s, r.blocks)
        ctx = np.empty(self.n_slots, np.int32)
        for s, r in enumerate(self.slots):
            r.ctx += 1
            r.budget -= 1
            ctx[s] = r.ctx
        return ctx


class StackEngine:
    """The GPU side: L layers (packed weights, K/V pools) and device copies of the tables.  A layer's pool is
    a (K, V) pair of BF16 tensors or an api.PoolF8; all layers have the same kind."""

    def __init__(self, api, cfgs, packed, pools, n_slots, max_blocks, max_prefill_tokens,
                 device="cuda"):
        self.api = api
        self.cfgs, self.packed, self.pools = cfgs, packed, pools
        self.n_slots = n_slots
        cfg = cfgs[0]
        self.H = cfg.hidden
        self.table = torch.full((n_slots, max_blocks), -1, dtype=torch.int32, device=device)
        self.ctx = torch.zeros(n_slots, dtype=torch.int32, device=device)
        self.f8 = isinstance(pools[0], api.PoolF8)
        self.ws = (api.new_workspace_f8 if self.f8 else api.new_workspace)(cfg, max(n_slots, max_prefill_tokens),
                                                                           max_blocks, device)
        self._blocks = None
        self.status = api.new_status(device)
        self.x = torch.zeros(n_slots, self.H, dtype=torch.bfloat16, device=device)
        self.bufs = [torch.empty(n_slots, self.H, dtype=torch.bfloat16, device=device) for _ in range(2)]
        self.pf_x = torch.empty(max_prefill_tokens, self.H, dtype=torch.bfloat16, device=device)
        self.pf_bufs = [torch.empty(max_prefill_tokens, self.H, dtype=torch.bfloat16, device=device)
                        for _ in range(2)]
        self.pf_pos = torch.empty(max_prefill_tokens, dtype=torch.int32, device=device)
        self.pf_table = torch.full((n_slots, max_blocks), -1, dtype=torch.int32, device=device)
        self.pf_ctx = torch.zeros(n_slots, dtype=torch.int32, device=device)
        self.graph = None
        self.y = None
        # the buffers are filled on the stream that is current here, and used on the caller's from now on
        torch.cuda.current_stream(self.table.device).synchronize()

    def prefill(self, n_req, prompt_len, stream):
        """All layers over the n_req requests whose rows are in pf_table[:n_req] and whose
        inputs are in pf_x[:n_req * prompt_len]; their positions in pf_pos (BF16 pools) or their
        context lengths, which count the prompt, in pf_ctx (e4m3 pools)."""
        T = n_req * prompt_len
        src = self.pf_x[:T]
        for l in range(len(self.cfgs)):
            dst = self.pf_bufs[l & 1][:T]
            if self.f8:
                self.api.layer_prefill_f8(self.cfgs[l], self.packed[l], src, self.pools[l], self.pf_table[:n_req],
                                          self.pf_ctx[:n_req], prompt_len, y=dst, workspace=self.ws,
                                          status=self.status, stream=stream)
                src = dst
                continue
            k, v = self.pools[l]
            self.api.layer_prefill(self.cfgs[l], self.packed[l], src, self.pf_pos[:T], n_req, prompt_len,
                                   k, v, self.pf_table[:n_req], y=dst, workspace=self.ws,
                                   status=self.status, stream=stream)
            src = dst
        return src

    def _decode_layers(self, stream):
        src = self.x
        for l in range(len(self.cfgs)):
            dst = self.bufs[l & 1]
            if self.f8:
                self.api.layer_decode_step_f8(self.cfgs[l], self.packed[l], src, self.pools[l], self.table, self.ctx,
                                              y=dst, workspace=self.ws, status=self.status, stream=stream)
                src = dst
                continue
            k, v = self.pools[l]
            self.api.layer_decode_step(self.cfgs[l], self.packed[l], src, k, v, self.table, self.ctx,
                                       y=dst, workspace=self.ws, status=self.status, stream=stream)
            src = dst
        return src

    @property
    def blocks(self):
        """Every layer's pool as one BlockSet, for copy_blocks and compact: the pools then have as many blocks each.
        (The layer calls take each layer's own pool, of any number of blocks.)"""
        if self._blocks is None:
            self._blocks = self.api.BlockSet([t for p in self.pools for t in (p.tensors() if self.f8 else p)])
        return self._blocks

    def copy_blocks(self, pairs, stream):
        """Copies blocks (from, to), as Scheduler.fork names them, in the pools of every layer."""
        if pairs:
            t = torch.tensor(pairs, dtype=torch.int32, device=self.table.device)
            stream.wait_stream(torch.cuda.current_stream(self.table.device))
            t.record_stream(stream)
            self.api.copy_blocks(self.blocks, t, status=self.status, stream=stream)

    def compact(self, scheduler: Scheduler, stream) -> int:
        """Packs the blocks of the scheduler's requests to the front of every pool, and renames them in the
        scheduler and in the device tables (a row of pf_table that belongs to no request any more becomes -1).
        Waits for the stream; returns the number of blocks moved.  A block that somebody besides the requests
        holds raises ValueError before anything is moved: to the plan it would be free, or its id would go stale."""
        held = scheduler.held_outside()
        if held:
            raise ValueError(f"blocks {held[:8]} are held outside the requests: free them before packing")
        blocks = self.blocks
        stream.wait_stream(torch.cuda.current_stream(self.table.device))
        with torch.cuda.stream(stream):                       # behind the steps that still read the table
            self.table.copy_(torch.from_numpy(scheduler.table))
            _, pairs, counts, block_map = self.api.compact_blocks(self.table, blocks.num_blocks,
                                                                  new_table=self.table, status=self.status)
            self.api.copy_blocks(blocks, pairs, n_pairs=counts[1:], status=self.status)
            old = self.pf_table
            known = (old >= 0) & (old < blocks.num_blocks)
            old.copy_(torch.where(known, block_map[torch.where(known, old, 0).long()], old))
            block_map, counts = block_map.cpu().numpy(), counts.tolist()
        scheduler.apply_map(block_map)
        return counts[1]

    def capture_decode(self, stream):
        """Records the all-layer decode step once as a CUDA graph (replayed by decode())."""
        with torch.cuda.stream(stream):
            self.y = self._decode_layers(stream)      # warm-up outside the capture
        stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            self.y = self._decode_layers(stream)
        self.graph = g

    def decode(self, stream):
        if self.graph is not None:
            with torch.cuda.stream(stream):
                self.graph.replay()
            return self.y
        self.y = self._decode_layers(stream)
        return self.y


def kv_blocks_needed(ctx_hi: int, n_slots: int, steps: int, prompt_len: int, block_size: int) -> int:
    """A pool size that covers the resident contexts, their growth over `steps` steps and
    the admitted requests' prompts, with head room for block rounding."""
    per_slot = -(-(ctx_hi + steps + prompt_len) // block_size) + 2
    return n_slots * per_slot


__all__ = ["BlockAllocator", "Request", "Scheduler", "StackEngine", "kv_blocks_needed"]
