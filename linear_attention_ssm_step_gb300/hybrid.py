"""A small hybrid decoder's layers on the library's serving calls: KDA layers and
attention layers over a paged cache, for requests that bring any number of new
tokens in a step (chunks of prompts, decode tokens, or none).

One step is: the page plan (kda_paged_plan), then layer by layer, on the packed
rows of all requests,
  a KDA layer         projections, kda_prefill on the request's state slot
  an attention layer  projections, kda_rope_append, kda_paged_attention, or on a
                      cache in 8 bits kda_rope_append_fp8, kda_paged_attention_fp8
each with an RMS norm before and a residual around it. Projections are plain
torch matrix products with random weights: this module shows how the calls are
used together, and is not a model.

    python -m linear_attention_ssm_step_gb300.hybrid
"""

import torch

from . import kda

HEAD_DIM = 128  # of KDA layers (the library's) and, here, of attention layers too


class HybridLayers:
    def __init__(self, hidden=1024, layers="kkka", heads=8, kv_heads=2, requests=4, pages=256, page_size=64,
                 max_tokens=4096, rope_base=10000.0, device="cuda", seed=0, cache_bits=16):
        """layers: one letter each, "k" KDA, "a" attention. requests: rows of the
        block table and slots of the KDA state; max_tokens: longest request;
        cache_bits: 16 (bf16) or 8 (E4M3 codes and scales) for keys and values."""
        if cache_bits not in (8, 16):
            raise ValueError(f"cache_bits must be 8 or 16, got {cache_bits}")
        self.cache_bits = cache_bits
        self.hidden, self.layers, self.heads, self.kv_heads = hidden, layers, heads, kv_heads
        self.page_size, self.pages, self.device = page_size, pages, torch.device(device)
        gen = torch.Generator(device=self.device).manual_seed(seed)

        def weight(rows, cols):
            w = torch.randn((rows, cols), generator=gen, device=self.device) * rows ** -0.5
            return w.to(torch.bfloat16)

        self.weights, self.memory = [], []
        for kind in layers:
            if kind == "k":
                # q, k, v, the gate's input (heads of 128 each) and beta's logits in one projection
                self.weights.append({"in": weight(hidden, heads * (4 * HEAD_DIM + 1)),
                                     "out": weight(heads * HEAD_DIM, hidden),
                                     "A_log": torch.rand(heads, generator=gen, device=self.device),
                                     "dt_bias": torch.randn((heads, HEAD_DIM), generator=gen, device=self.device)})
                self.memory.append(torch.zeros((requests, heads, HEAD_DIM, HEAD_DIM), dtype=torch.bfloat16,
                                               device=self.device))
            else:
                self.weights.append({"in": weight(hidden, (heads + 2 * kv_heads) * HEAD_DIM),
                                     "out": weight(heads * HEAD_DIM, hidden)})
                if cache_bits == 8:  # k_codes, v_codes, k_scales, v_scales
                    self.memory.append(kda.paged_fp8_cache(pages, page_size, kv_heads, HEAD_DIM, self.device))
                else:  # keys and values of a page side by side
                    self.memory.append(torch.zeros((pages, 2, page_size, kv_heads, HEAD_DIM), dtype=torch.bfloat16,
                                                   device=self.device))
        int32 = {"dtype": torch.int32, "device": self.device}
        self.slots = torch.arange(requests, **int32)
        self.cached = torch.zeros(requests, **int32)
        self.block_table = torch.full((requests, -(-max_tokens // page_size)), -1, **int32)
        self.free_pages = torch.arange(pages, **int32)
        self.free_count = torch.tensor([pages], **int32)
        self.error_word = torch.zeros(1, **int32)
        self.freqs = kda.rope_freqs(HEAD_DIM, rope_base, device=self.device)
        self.workspace = kda.paged_attention_workspace(HEAD_DIM, self.device)

    @staticmethod
    def _norm(x):
        y = x.float()
        return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def step(self, x, new_len):
        """x: bf16 [sum(new_len), hidden], the packed rows of all requests (request r's new_len[r] rows after those of
        the requests before it). Returns the layers' output rows; every request's state and cache move on, but for
        requests that the plan turns down (error_word says why): they stay as they were, and their rows mean nothing."""
        T, H, D = x.shape[0], self.heads, HEAD_DIM
        new_len = torch.tensor(new_len, dtype=torch.int32, device=self.device)
        plan = kda.kda_paged_plan(self.cached, new_len, self.block_table, self.free_pages, self.free_count,
                                  self.page_size, self.pages, T, error_word=self.error_word)
        # the kv_len of a request turned down is 0 (as is the sum for a negative length that takes all of the cached away)
        admitted = (new_len >= 0) & (plan.kv_len == self.cached + new_len)
        slots = torch.where(admitted, self.slots, -1)
        for kind, w, memory in zip(self.layers, self.weights, self.memory):
            y = self._norm(x) @ w["in"]
            if kind == "k":
                q, k, v, g = (y[:, i * H * D:(i + 1) * H * D].view(T, H, D) for i in range(4))
                out = kda.kda_prefill(memory, slots, plan.cu_new, q, k, v, g, y[:, 4 * H * D:], w["A_log"],
                                      w["dt_bias"], error_word=self.error_word)
            else:
                q, k, v = y.view(T, -1, D).split((H, self.kv_heads, self.kv_heads), dim=1)
                if self.cache_bits == 8:
                    append, attention, cache = kda.kda_rope_append_fp8, kda.kda_paged_attention_fp8, memory
                else:
                    append, attention, cache = kda.kda_rope_append, kda.kda_paged_attention, (memory[:, 0], memory[:, 1])
                append(q, k, v, plan.positions, plan.slots, self.freqs, *cache, q_out=q, error_word=self.error_word)
                out = attention(q, *cache, self.block_table, plan.cu_new, plan.kv_len, workspace=self.workspace,
                                error_word=self.error_word)
            x = x + out.reshape(T, H * D) @ w["out"]
        self.cached, self.free_count = torch.where(admitted, plan.kv_len, self.cached), plan.free_count
        return x

    def cached_rows(self, layer):
        """Keys and values that an attention layer has cached, request after request: bf16 [sum of cached, kv_heads,
        128] each, to be moved elsewhere or looked at."""
        memory = self.memory[layer]
        if self.layers[layer] != "a":
            raise ValueError(f"layer {layer} is no attention layer")
        lengths = self.cached.tolist()
        total = sum(lengths)
        if self.cache_bits == 8:
            starts = torch.zeros(len(lengths) + 1, dtype=torch.int32, device=self.device)
            starts[1:] = self.cached.cumsum(0)
            return kda.kda_paged_read_fp8(*memory, self.block_table, starts, self.cached, total, error_word=self.error_word)
        rows = [memory[self.block_table[r, :-(-n // self.page_size)].long()].transpose(0, 1).flatten(1, 2)[:, :n]
                for r, n in enumerate(lengths)]
        return kda.PagedRead(*torch.cat(rows, dim=1))


def main():
    model = HybridLayers()
    gen = torch.Generator(device=model.device).manual_seed(1)
    for new in ([512, 100, 0, 7], [512, 1, 300, 1], [1, 1, 1, 1], [1, 1, 1, 1]):
        x = torch.randn((sum(new), model.hidden), generator=gen, device=model.device).to(torch.bfloat16)
        y = model.step(x, new)
        print(f"new tokens {new}: {tuple(y.shape)} rows, tokens cached {model.cached.tolist()}, "
              f"free pages {int(model.free_count)}, error word {int(model.error_word)}")


if __name__ == "__main__":
    main()
