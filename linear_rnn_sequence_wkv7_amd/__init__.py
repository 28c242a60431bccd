"""MI355X-native RWKV-7 WKV recurrence and the operators around it: HIP kernels
behind a C-ABI library.

Submodules:
  inputs    -- seeded synthetic inputs (numpy only)
  wkv7      -- ctypes binding over libwkv7.so (torch supplies device memory and streams)
  ssm       -- the same for the selective state space scan (prompt, step, backward)
  shortconv -- the short causal convolution in front of a recurrence
  groupnorm -- the group norm, activation and gate behind one
  layernorm -- the layer norm in front of one, with the residual stream's sum
  linattn   -- linear attention with a decay for each head (prompt, step, backward)
"""
__all__ = ["inputs", "wkv7", "ssm", "shortconv", "groupnorm", "layernorm", "linattn"]
