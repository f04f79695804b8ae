// Operators between the encoder and a language model, on packed ids: block
// plans of a paged cache (blocks.cuh), embedding lookup and its gradient
// (embed.cuh), penalties, biases and grammar masks on logits (logits.cuh).
// The source pages end at the ids; these have no counterpart there.
//
// They share the handle's device, workspace and status with the encoder
// (handle.cuh). No kernel waits on another CTA outside its own cluster.

#include "ops.cuh"
#include "vec.cuh"
#include "blocks.cuh"
#include "embed.cuh"
#include "logits.cuh"
