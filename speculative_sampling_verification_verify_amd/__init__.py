"""MI355X (gfx950) batched speculative-sampling verify step.

The compute path is the HIP library ``libspecverify.so`` (built from
``csrc/``); ``binding`` marshals torch tensors into its C ABI.  ``logits`` does
the same for ``libspeclogits.so``, the operators between a model and these
calls: logits from a 4-bit head, penalties, biases and grammar masks, and the
token history.  ``synth`` makes seeded synthetic inputs.  Importing this
package does not load the libraries; the first call into ``binding`` or
``logits`` does, and fails loudly when one is missing."""
