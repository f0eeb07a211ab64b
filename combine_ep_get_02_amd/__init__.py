"""MI355X-native expert-parallel dispatch/combine core (one GPU's share).

The four stages -- layout, notify, dispatch, combine -- are HIP kernels for
gfx950 behind the C ABI declared in ``include/ep.h`` (library ``libep.so``).
``combine_ep_get_02_amd.ep`` is the thin ctypes binding over that ABI;
``include/ep_experts.h`` and ``combine_ep_get_02_amd.experts`` are the steps of
an expert layer on either side of them: the router, the experts' E4M3 products
and the combine of grouped rows, with the gradients of the first and the last.
``combine_ep_get_02_amd.inputs`` draws the seeded synthetic workloads.
"""
