/* Sizes and field offsets of the output head's and the moments' structs of
 * mfsdp.h as a C compiler sees them, one "name value" per line. */
#include <stddef.h>
#include <stdio.h>

#include "mfsdp.h"

#define SZ(t) printf("sizeof:%s %zu\n", #t, sizeof(t))
#define OF(t, f) printf("offsetof:%s.%s %zu\n", #t, #f, offsetof(t, f))

int main(void) {
    SZ(mfsdp_moments_args);
    OF(mfsdp_moments_args, state); OF(mfsdp_moments_args, first); OF(mfsdp_moments_args, second);
    OF(mfsdp_moments_args, type); OF(mfsdp_moments_args, stream);
    SZ(mfsdp_head_record);
    OF(mfsdp_head_record, max); OF(mfsdp_head_record, sum); OF(mfsdp_head_record, wsum);
    OF(mfsdp_head_record, target); OF(mfsdp_head_record, found); OF(mfsdp_head_record, active);
    SZ(mfsdp_head_logprob_args);
    OF(mfsdp_head_logprob_args, params); OF(mfsdp_head_logprob_args, x); OF(mfsdp_head_logprob_args, n);
    OF(mfsdp_head_logprob_args, x_stride); OF(mfsdp_head_logprob_args, x_type); OF(mfsdp_head_logprob_args, id_type);
    OF(mfsdp_head_logprob_args, ids); OF(mfsdp_head_logprob_args, first_id); OF(mfsdp_head_logprob_args, scale);
    OF(mfsdp_head_logprob_args, top_k); OF(mfsdp_head_logprob_args, records); OF(mfsdp_head_logprob_args, logp);
    OF(mfsdp_head_logprob_args, entropy); OF(mfsdp_head_logprob_args, top_ids); OF(mfsdp_head_logprob_args, top_logp);
    OF(mfsdp_head_logprob_args, top_logits); OF(mfsdp_head_logprob_args, workspace);
    OF(mfsdp_head_logprob_args, workspace_bytes); OF(mfsdp_head_logprob_args, stream);
    SZ(mfsdp_head_total_args);
    OF(mfsdp_head_total_args, parts); OF(mfsdp_head_total_args, count); OF(mfsdp_head_total_args, n);
    OF(mfsdp_head_total_args, records); OF(mfsdp_head_total_args, logp); OF(mfsdp_head_total_args, entropy);
    OF(mfsdp_head_total_args, part_top_ids); OF(mfsdp_head_total_args, part_top_logits);
    OF(mfsdp_head_total_args, top_ids); OF(mfsdp_head_total_args, top_logp); OF(mfsdp_head_total_args, top_logits);
    OF(mfsdp_head_total_args, top_k); OF(mfsdp_head_total_args, stream);
    SZ(mfsdp_head_grad_args);
    OF(mfsdp_head_grad_args, params); OF(mfsdp_head_grad_args, x); OF(mfsdp_head_grad_args, n);
    OF(mfsdp_head_grad_args, x_stride); OF(mfsdp_head_grad_args, x_type); OF(mfsdp_head_grad_args, id_type);
    OF(mfsdp_head_grad_args, ids); OF(mfsdp_head_grad_args, first_id); OF(mfsdp_head_grad_args, scale);
    OF(mfsdp_head_grad_args, accumulate); OF(mfsdp_head_grad_args, records); OF(mfsdp_head_grad_args, dlogp);
    OF(mfsdp_head_grad_args, dentropy); OF(mfsdp_head_grad_args, dx); OF(mfsdp_head_grad_args, dx_stride);
    OF(mfsdp_head_grad_args, grads); OF(mfsdp_head_grad_args, workspace); OF(mfsdp_head_grad_args, workspace_bytes);
    OF(mfsdp_head_grad_args, stream);
    return 0;
}
