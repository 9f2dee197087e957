"""A small hybrid model served with the library: recurrent-state (KDA) layers and latent attention
layers in turn, prompts prefilled, tokens decoded, answers reported with their log probabilities.

    python examples/hybrid_serving_step.py

Random weights; the projections are torch matrix products, as an engine would run its own.  Per layer
kind the calls are
  KDA      kda_chunk_prefill for prompts, kda_recurrent_decode for a token, one state slot a request
  latent   kda_latent_append into a paged cache, kda_latent_prefill (expanded keys and values) for
           prompts, kda_latent_decode (absorbed projections) for a token
and kda_token_logprobs after the output projection.  Everything of a decode step runs on one stream
without a host wait.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import serving_kda_chunk_gb300 as kda  # noqa: E402

D, H, VOCAB, LAYERS, PAGE = 256, 4, 1003, 4, 16  # model width, heads, vocabulary, layers, tokens a page
NOPE, ROPE, LATENT = 128, 64, 512
SCALE = 1 / math.sqrt(NOPE + ROPE)


def norm(x):
    return torch.nn.functional.rms_norm(x, (x.shape[-1],))


class Model:
    def __init__(self, requests, max_tokens, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def w(*shape):
            return (torch.randn(*shape, generator=g, device=device) / math.sqrt(shape[-2])).to(dtype)

        self.R, self.dtype, self.device = requests, dtype, device
        self.embed = torch.randn(VOCAB, D, generator=g, device=device).to(dtype)
        self.head = w(D, VOCAB)
        self.layers = []
        pages = -(-max_tokens // PAGE)
        for i in range(LAYERS):
            if i % 2 == 0:
                self.layers.append(dict(
                    kind="kda", qkvg=w(D, 4 * H * 128), beta=w(D, H), out=w(H * 128, D),
                    pool=torch.zeros(requests, H, 128, 128, device=device)))
            else:
                up = w(H, LATENT, NOPE + 128)  # latent vector -> a head's key and value
                self.layers.append(dict(
                    kind="latent", q=w(D, H * (NOPE + ROPE)), kv=w(D, LATENT + ROPE), up=up,
                    up_flat=up.transpose(0, 1).reshape(LATENT, -1).contiguous(),
                    norm=torch.ones(LATENT, dtype=dtype, device=device), out=w(H * 128, D),
                    cache=torch.zeros(requests * pages, PAGE, LATENT + ROPE, dtype=dtype, device=device)))
        # request r's tokens lie in pages r * pages ..; an engine's allocator would hand pages out
        self.table = torch.arange(requests * pages, device=device, dtype=torch.int32).view(requests, pages)
        self.pages = pages
        self.length = torch.zeros(requests, dtype=torch.int32, device=device)
        self.slot = torch.arange(requests, device=device, dtype=torch.int32)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.workspace = torch.empty(kda.kda_latent_decode_workspace_size(requests, 1, H), dtype=torch.uint8,
                                     device=device)

    def _places(self, request, position):
        page = self.table[request.long(), (position // PAGE).long()]
        return (page * PAGE + position % PAGE).to(torch.int32)

    def _kda_inputs(self, layer, x):
        q, k, v, gate = (t.contiguous() for t in (x @ layer["qkvg"]).view(-1, 4, H, 128).unbind(1))
        return q, k, v, x @ layer["beta"], gate

    def _append(self, layer, x, places):
        kv = x @ layer["kv"]
        kda.kda_latent_append(kv, layer["cache"], places, weight=layer["norm"], dev_status=self.status)

    def prefill(self, prompts):
        """Logits of every prompt position; states and caches hold the prompts afterwards."""
        lens = [len(p) for p in prompts]
        cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=self.device)
        tokens = torch.tensor([t for p in prompts for t in p], device=self.device)
        T = tokens.numel()
        request = torch.repeat_interleave(torch.arange(self.R, device=self.device), torch.tensor(lens, device=self.device))
        position = torch.arange(T, device=self.device) - cu[request].long()
        places = self._places(request, position)
        x = self.embed[tokens]
        for layer in self.layers:
            y = norm(x)
            o = torch.empty(T, H, 128, dtype=self.dtype, device=self.device)
            if layer["kind"] == "kda":
                ws = torch.empty(kda.kda_chunk_prefill_workspace_size(T, self.R, H), dtype=torch.uint8, device=self.device)
                kda.kda_chunk_prefill(*self._kda_inputs(layer, y), cu, o, state_pool=layer["pool"],
                                      final_slot=self.slot, scale=128 ** -0.5, flags=kda.KDA_QK_L2NORM,
                                      workspace=ws, dev_status=self.status)
            else:
                self._append(layer, y, places)
                rows = layer["cache"].view(-1, LATENT + ROPE)[places.long()]
                up = (rows[:, :LATENT] @ layer["up_flat"]).view(T, H, NOPE + 128)
                kda.kda_latent_prefill((y @ layer["q"]).view(T, H, NOPE + ROPE), up[..., :NOPE], rows[:, LATENT:],
                                       up[..., NOPE:], cu, cu, o, scale=SCALE, dev_status=self.status)
            x = x + o.view(T, -1) @ layer["out"]
        self.length.copy_(torch.tensor(lens, device=self.device))
        return norm(x) @ self.head, cu

    def decode(self, tokens):
        """One token of every request: logits [R, VOCAB]."""
        R = self.R
        places = self._places(torch.arange(R, device=self.device), self.length.long())
        self.length += 1
        x = self.embed[tokens.long()]
        for layer in self.layers:
            y = norm(x)
            if layer["kind"] == "kda":
                o = torch.empty(R, H, 128, dtype=self.dtype, device=self.device)
                kda.kda_recurrent_decode(*self._kda_inputs(layer, y), layer["pool"], self.slot, o,
                                         scale=128 ** -0.5, flags=kda.KDA_QK_L2NORM, dev_status=self.status)
            else:
                self._append(layer, y, places)
                q = (y @ layer["q"]).view(R, H, NOPE + ROPE)
                # absorbed: the key up-projection into the query, the value one out of the output; both
                # batched over heads, whose layout the call takes as it is
                ql = torch.bmm(q[..., :NOPE].transpose(0, 1), layer["up"][..., :NOPE].transpose(1, 2)).transpose(0, 1)
                ol = torch.empty(H, R, LATENT, dtype=self.dtype, device=self.device).transpose(0, 1)
                kda.kda_latent_decode(ql, q[..., NOPE:], layer["cache"], self.table, self.length, ol, self.workspace,
                                      scale=SCALE, dev_status=self.status)
                o = torch.bmm(ol.transpose(0, 1), layer["up"][..., NOPE:]).transpose(0, 1)
            x = x + o.reshape(R, -1) @ layer["out"]
        return norm(x) @ self.head


def logprobs(logits, tokens, top=5):
    """(log probability, entropy, top ids, their log probabilities) of each row."""
    R = logits.shape[0]
    lp, ent = (torch.empty(R, device=logits.device) for _ in range(2))
    ids = torch.empty(R, top, dtype=torch.int32, device=logits.device)
    tl = torch.empty(R, top, device=logits.device)
    kda.kda_token_logprobs(logits, tokens, lp, entropy=ent, top_ids=ids, top_logprobs=tl)
    return lp, ent, ids, tl


def main(steps=8):
    prompts = [[(7 * i + 3 * j) % VOCAB for j in range(n)] for i, n in enumerate((5, 33, 70, 150))]
    model = Model(len(prompts), max_tokens=160 + steps)
    logits, cu = model.prefill(prompts)
    # the prompts' own log probabilities: each position predicts the next token
    ends = cu[1:].long() - 1
    rows = torch.ones(logits.shape[0], dtype=torch.bool, device=logits.device)
    rows[ends] = False
    following = torch.tensor([t for p in prompts for t in p[1:]], dtype=torch.int32, device=logits.device)
    lp, _, _, _ = logprobs(logits[rows], following)
    print("prompt tokens %d, mean log probability %.3f" % (sum(map(len, prompts)), lp.mean().item()))
    last = logits[ends]
    for step in range(steps):
        _, ent, ids, tl = logprobs(last, torch.full((len(prompts),), -1, dtype=torch.int32, device=logits.device))
        token = ids[:, 0].contiguous()
        print("step %d: tokens %s, log probabilities %s, entropies %s" % (
            step, token.tolist(), [round(v, 3) for v in tl[:, 0].tolist()], [round(v, 2) for v in ent.tolist()]))
        last = model.decode(token)
    assert int(model.status) == 0, "status %d" % int(model.status)


if __name__ == "__main__":
    main()
