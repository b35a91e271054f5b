"""GB300-native forward pass of the Test-Time-Training (TTT) layer.

The compute path is the CUDA library ``libttt.so`` (C ABI in ``include/ttt.h``);
``abi`` is its Python binding, ``rotary`` makes the tables of ``abi.ttt_rope`` and
``synth`` is the seeded synthetic-input generator.
"""
from .abi import (TTTError, ttt_block_norm_bwd, ttt_block_norm_fwd,  # noqa: F401
                  ttt_launch_count, ttt_linear_fwd, ttt_mlp_fwd, ttt_recurrence_bwd, ttt_recurrence_fwd, ttt_rope,
                  ttt_sync_status)
from .rotary import rope_table  # noqa: F401
