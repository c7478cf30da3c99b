"""GB300-native weight-only quantized dequant-GEMV (INT8 per tensor and
outlier-aware INT4), a C-ABI CUDA library (libqz) with a thin Python API."""
from .api import *  # noqa: F401,F403
from .api import Int4oMatrix, Int8Matrix, Pager, QzError  # noqa: F401
from .layer import (LoraAdapters, PagedKV, PagedKVInt8, SeqBatch, attention_paged,  # noqa: F401
                    attention_workspace, cache_read, lora, lora_workspace, rmsnorm, rmsnorm_int8,
                    rope_append, rope_table, sample)
