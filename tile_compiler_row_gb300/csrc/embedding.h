// Launchers of the embedding lookup and its gradient (embedding.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace tile {

struct EmbeddingArgs {
    const long long *tokens;   // [rows]
    const void *weight;        // lookup: [vocab][width]
    void *out;                 // lookup: [rows][width]
    const void *dout;          // gradient: [rows][width]
    void *dweight;             // gradient: [vocab][width]
    long long ignore;
    int rows, width, vocab;
    float scale;
    bool add;                  // dweight += instead of =
    void *ws;
    unsigned int *status;
};

// vectors: every matrix is 16-byte aligned and rows are whole 16-byte vectors
cudaError_t launch_embedding(int elem, bool vectors, EmbeddingArgs a, cudaStream_t stream);
size_t embedding_backward_workspace(int rows, int width, int vocab);
cudaError_t launch_embedding_backward(int elem, int into, bool vectors, EmbeddingArgs a,
                                      cudaStream_t stream);

}  // namespace tile
