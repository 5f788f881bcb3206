"""GB300-native per-block KV-cache token eviction (KNorm, Q-Filters, CurDKV-adapted).

The compute path is the C-ABI library ``libevict.so`` built from ``csrc/``;
``binding`` marshals arguments to it. Importing this package does not load
the library; ``binding.load()`` does, and raises if it is missing. ``paged``
holds the steps around a kept cache: rotary positions, pages of a batch's
own rows, and attention over a shared kept prefix and those pages.
"""
__all__ = ["binding", "paged", "synth"]
