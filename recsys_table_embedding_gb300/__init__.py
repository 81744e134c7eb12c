"""GB300-native table-batched embedding (TBE) training hot path.

The compute lives in libtbe_gb300.so (hand-written CUDA for sm_103a behind
the C ABI in include/tbe.h); ``tbe`` is its ctypes binding, ``tokens`` the
binding of the token operators.
"""
from .tbe import (TBE, Batch, Meta, Tables, TbeError, config, lib, meta_view, tbe_backward_rowwise_adagrad,
                  tbe_forward, tbe_meta_bind, tbe_preprocess, tbe_preprocess_static, tbe_query_sizes,
                  tbe_select_path)
from .tokens import (Route, tbe_distill_backward, tbe_distill_forward, tbe_distill_loss_grad,
                     tbe_route_combine, tbe_route_combine_backward, tbe_route_dispatch,
                     tbe_route_dispatch_backward, tbe_route_sort, tbe_route_sort_dispatch,
                     tbe_token_backward, tbe_token_forward)

__all__ = ["TBE", "Batch", "Meta", "Tables", "TbeError", "config", "lib", "meta_view",
           "tbe_backward_rowwise_adagrad", "tbe_forward", "tbe_meta_bind", "tbe_preprocess",
           "tbe_preprocess_static",
           "tbe_query_sizes", "tbe_select_path",
           "Route", "tbe_distill_backward", "tbe_distill_forward", "tbe_distill_loss_grad",
           "tbe_route_combine", "tbe_route_combine_backward", "tbe_route_dispatch",
           "tbe_route_dispatch_backward", "tbe_route_sort", "tbe_route_sort_dispatch",
           "tbe_token_backward", "tbe_token_forward"]
