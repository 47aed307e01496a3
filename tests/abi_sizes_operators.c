/* Sizes and field offsets of the gradient and embedding structs of mfsdp.h as
 * a C compiler sees them, one "name value" per line. */
#include <stddef.h>
#include <stdio.h>

#include "mfsdp.h"

#define SZ(t) printf("sizeof:%s %zu\n", #t, sizeof(t))
#define OF(t, f) printf("offsetof:%s.%s %zu\n", #t, #f, offsetof(t, f))

int main(void) {
    SZ(mfsdp_grad_stats);
    OF(mfsdp_grad_stats, sumsq); OF(mfsdp_grad_stats, norm); OF(mfsdp_grad_stats, scale);
    SZ(mfsdp_grad_norm_args);
    OF(mfsdp_grad_norm_args, grads); OF(mfsdp_grad_norm_args, workspace); OF(mfsdp_grad_norm_args, workspace_bytes);
    OF(mfsdp_grad_norm_args, max_norm); OF(mfsdp_grad_norm_args, eps); OF(mfsdp_grad_norm_args, stats);
    OF(mfsdp_grad_norm_args, entry_norms); OF(mfsdp_grad_norm_args, stream); OF(mfsdp_grad_norm_args, flags);
    SZ(mfsdp_grad_clip_args);
    OF(mfsdp_grad_clip_args, grads); OF(mfsdp_grad_clip_args, out); OF(mfsdp_grad_clip_args, scale);
    OF(mfsdp_grad_clip_args, workspace); OF(mfsdp_grad_clip_args, workspace_bytes);
    OF(mfsdp_grad_clip_args, stream); OF(mfsdp_grad_clip_args, flags);
    SZ(mfsdp_embed_lookup_args);
    OF(mfsdp_embed_lookup_args, params); OF(mfsdp_embed_lookup_args, ids); OF(mfsdp_embed_lookup_args, n_ids);
    OF(mfsdp_embed_lookup_args, id_type); OF(mfsdp_embed_lookup_args, out_type);
    OF(mfsdp_embed_lookup_args, first_id); OF(mfsdp_embed_lookup_args, out);
    OF(mfsdp_embed_lookup_args, out_stride); OF(mfsdp_embed_lookup_args, scale); OF(mfsdp_embed_lookup_args, stream);
    SZ(mfsdp_embed_grad_args);
    OF(mfsdp_embed_grad_args, grads); OF(mfsdp_embed_grad_args, ids); OF(mfsdp_embed_grad_args, n_ids);
    OF(mfsdp_embed_grad_args, id_type); OF(mfsdp_embed_grad_args, dout_type); OF(mfsdp_embed_grad_args, first_id);
    OF(mfsdp_embed_grad_args, dout); OF(mfsdp_embed_grad_args, dout_stride); OF(mfsdp_embed_grad_args, scale);
    OF(mfsdp_embed_grad_args, accumulate); OF(mfsdp_embed_grad_args, workspace);
    OF(mfsdp_embed_grad_args, workspace_bytes); OF(mfsdp_embed_grad_args, stream);
    return 0;
}
