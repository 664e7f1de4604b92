"""Programmatic dependent launch: the forward path's kernels are launched so that each may set up
(barriers, TMEM, tensor-map prefetch) while the previous kernel on the stream drains, and wait
for that kernel's completion before touching memory.  A rollout run that way (eager calls and
CUDA-graph replays) must give exactly the results of plain launches (MLA_NO_PDL=1), which this
test runs in a child process since the library reads the switch once per process."""
import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys
import numpy as np
import torch
from mla_latent_kv_attn_b200 import api, inputs, rollout

cfg = inputs.small_bf16_config()
c = api.make_config(cfg)
w = rollout.upload_weights(c, inputs.layer_weights(cfg, 0))
ring, buf = rollout.Ring(c), rollout.ChunkBuffers(c)
outs, lses = [], []
for ch in range(cfg.n_chunks):
    buf.x.copy_(torch.from_numpy(inputs.chunk_x(cfg, ch)).to(torch.bfloat16))
    if ch < 2:
        o = rollout.run_chunk(c, w, ring, buf, ch, fused_q=True)
    else:
        o = rollout.ChunkGraph(c, w, ring, buf, ch, fused_q=True).replay()
    outs.append(o.float().cpu().numpy())
    lses.append(buf.lse.cpu().numpy())
torch.cuda.synchronize()
rollout.check_device_status(buf)
np.savez(sys.argv[1], o=np.stack(outs), lse=np.stack(lses), cache=ring.cache.float().cpu().numpy(),
         slot_frame=ring.slot_frame.cpu().numpy())
"""


def _run(path, extra_env):
    env = {k: v for k, v in os.environ.items() if k != "MLA_NO_PDL"}
    env.update(extra_env)
    env["PYTHONPATH"] = ROOT + os.pathsep + env.get("PYTHONPATH", "")
    r = subprocess.run([sys.executable, "-c", CHILD, str(path)], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    return np.load(path)


def test_programmatic_and_plain_launches_agree(tmp_path):
    a = _run(tmp_path / "pdl.npz", {})
    b = _run(tmp_path / "plain.npz", {"MLA_NO_PDL": "1"})
    for k in ("o", "lse", "cache", "slot_frame"):
        assert np.array_equal(a[k], b[k]), k


CROSS_CHILD = r"""
import sys
import numpy as np
import torch
from mla_latent_kv_attn_b200 import api, inputs, rollout

outs = {}
g = torch.Generator(device="cuda").manual_seed(1)
new = lambda *shape: torch.randn(shape, generator=g, device="cuda").bfloat16()
for n, (B, n_q, n_kv, H, Hkv, d, lens) in enumerate((
        (1, 700, 300, 4, 4, 128, [300]), (3, 260, 333, 8, 2, 64, [333, 0, 130]),
        (4, 90, 300, 40, 40, 128, [300, 1, 0, 200]), (2, 9, 129, 3, 1, 64, [129, 5]))):
    q, k, v, grad = new(B, n_q, H, d), new(B, n_kv, Hkv, d), new(B, n_kv, Hkv, d), new(B, n_q, H, d)
    text = rollout.EncoderStates(k, v, n_heads=H,
                                 kv_len=torch.tensor(lens, device="cuda", dtype=torch.int32))
    out, lse = torch.empty_like(q), torch.empty((B, H, n_q), device="cuda")
    grads = [torch.empty_like(t) for t in (q, k, v)]
    for _ in range(3):                       # back to back, into the same outputs and workspace
        text.attend(q, out, lse=lse)
        text.backward(q, out, lse, grad, *grads)
    for name, t in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        outs[f"{name}{n}"] = t.float().cpu().numpy()
    assert int(text.dev_status) == 0
cfg = inputs.small_bf16_config()
c = api.make_config(cfg)
w = rollout.upload_weights(c, inputs.layer_weights(cfg, 0))
ring, buf = rollout.RingQ4(c), rollout.ChunkBuffers(c, q4=True)
for ch in range(cfg.n_chunks):
    buf.x.copy_(torch.from_numpy(inputs.chunk_x(cfg, ch)).to(torch.bfloat16))
    outs[f"o{ch}"] = rollout.run_chunk(c, w, ring, buf, ch).float().cpu().numpy()
rollout.check_device_status(buf)
outs["values"] = ring.read().float().cpu().numpy()
np.savez(sys.argv[1], **outs)
"""


def test_cross_attention_and_the_4_bit_ring_agree_too(tmp_path, monkeypatch):
    monkeypatch.setitem(globals(), "CHILD", CROSS_CHILD)
    a = _run(tmp_path / "pdl.npz", {})
    b = _run(tmp_path / "plain.npz", {"MLA_NO_PDL": "1"})
    assert len(a.files) == 5 * 4 + 4 + 1
    for k in a.files:
        assert np.array_equal(a[k], b[k]), k
