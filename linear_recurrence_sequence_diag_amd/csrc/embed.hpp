// embed.hpp -- host-side launchers of the embedding lookup and of its gradient
// (internal to liblrscan).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace lrscan {

struct EmbedShape {
    int64_t N, V, D;  // tokens, table rows, row length
    int id_bytes;     // 4 or 8
    int dtype;        // DT_F32 / DT_BF16
};

bool embed_fits(const EmbedShape& s);
hipError_t launch_embed_fwd(const EmbedShape& s, const void* ids, const void* w, float scale, void* out,
                            hipStream_t st);

// Whether a gradient sorts its tokens; only then is its workspace used.
bool embed_sorts(const EmbedShape& s);

// `ws` holds embed_ws_bytes (256-byte aligned; NULL where nothing is sorted).
// `add`: rows that tokens name are added to and the others left as they are;
// else every row is written.
size_t embed_ws_bytes(const EmbedShape& s);
hipError_t launch_embed_bwd(const EmbedShape& s, const void* ids, const void* g, float scale,
                            void* grad, int grad_dtype, bool add, void* ws, hipStream_t st);

}  // namespace lrscan
